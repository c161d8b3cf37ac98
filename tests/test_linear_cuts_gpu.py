"""Linear attention where sequences are cut into segments, packed in large numbers, or asked for without their last state.

Bounds as in test_linear_gpu.py and test_linear_bwd_gpu.py, but for a decay's gradient: within a chunk of 128 tokens it is a
running sum of differences, every partial sum of which is a difference of two of the chunk's gradients (each at most the
chunk's largest mass), so what the chunk's running sum is off by goes by that mass, not by the sequence's."""
import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from linear_cases import absolute, backward, close, forward, inputs
from test_linear_gpu import FINE, check_forward, half, on_gpu, packed_case, sequence

pytestmark = pytest.mark.gpu


def check_backward(x, g, scale=1.0):
    ref, mass = backward(**x, scale=scale), backward(**absolute(x), scale=abs(scale))
    for n in ("q", "k", "v"):
        close(g[n], ref[n], mass[n], 2.0 ** -8 + FINE, 2.0 ** -8, n)
    m = mass["log_alpha"]
    T = m.shape[1]
    chunks = torch.nn.functional.pad(m, (0, 0, 0, -T % 128)).unflatten(1, (-1, 128)).amax(2, keepdim=True)
    near = chunks.expand(-1, -1, 128, -1).flatten(1, 2)[:, :T]
    close(g["log_alpha"], ref["log_alpha"], m + 2.0 ** -17 / (2.0 ** -7 + FINE) * near, 2.0 ** -7 + FINE, half(g["log_alpha"].dtype),
          "log_alpha")
    close(g["initial_state"], ref["initial_state"], mass["initial_state"], FINE, 2.0 ** -24, "initial_state")


def with_gradients(lens, H, d, kind, seed):
    x = packed_case(lens, H, d, kind, seed)
    x["d_out"] = inputs((sum(lens),), H, d, kind, seed + 1, ("v",))["v"].cuda()
    x["d_final"] = torch.randn_like(x["state"])
    return x


def gradients(x, **kw):
    return kda.kda_linear_bwd(x["q"], x["k"], x["v"], x["log_alpha"], x["d_out"], initial_state=x["state"], d_final_state=x["d_final"],
                              cu_seqlens=x["cu"], **kw)


# the lengths of the second end with a segment (512 tokens here: 16 of them); a decay's range of a token or of thousands
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["slow", "mixed"])
@pytest.mark.parametrize("lens", [[1, 4100, 0, 700, 2, 9000, 129], [4096, 4096], [0, 6000, 0]])
def test_packed_gradients_through_segments(lens, kind, d):
    x = with_gradients(lens, 2, d, kind, 71)
    g = gradients(x, scale=0.7)
    for n, L in enumerate(lens):
        y, rows = sequence(x, n, lens)
        y["d_out"], y["d_final"] = x["d_out"][rows][None], x["d_final"][n:n + 1]
        part = {m: g[m][rows][None] for m in ("q", "k", "v", "log_alpha")}
        part["initial_state"] = g["initial_state"][n:n + 1]
        if L:
            check_backward(y, part, 0.7)
        else:
            assert torch.equal(part["initial_state"], y["d_final"])
    again = gradients(x, scale=0.7)
    for n in g:
        assert torch.equal(g[n], again[n]), n
    assert kda.kda_last_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_large_states_at_either_end_of_a_long_sequence(d):
    """Chunks that the states have faded from are held to their own mass."""
    T, H = 3000, 2
    x = on_gpu(inputs((1, T), H, d, "slow", 72, ("q", "k", "v", "d_out")))
    x["log_alpha"] = torch.full((1, T, H), -0.03, device="cuda").to(torch.bfloat16)
    x["state"], x["d_final"] = (1e4 * torch.randn((1, H, d, d), device="cuda") for _ in range(2))
    g = kda.kda_linear_bwd(x["q"], x["k"], x["v"], x["log_alpha"], x["d_out"], initial_state=x["state"], d_final_state=x["d_final"])
    check_backward(x, g)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,H", [(1, 5000, 2), (2, 2600, 3), (1, 4096, 4)])
def test_long_prompts_of_narrow_heads(B, T, H, out_dtype):
    x = on_gpu(inputs((B, T), H, 64, "mixed", 73))
    x["state"] = torch.randn((B, H, 64, 64), device="cuda")
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], out_dtype=out_dtype)
    check_forward(x, out, state, "mixed", 1.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [9, 300, 3000])
def test_outputs_without_the_last_state(T, out_dtype, d):
    x = on_gpu(inputs((2, T), 3, d, "mixed", 74))
    x["state"] = torch.randn((2, 3, d, d), device="cuda")
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], out_dtype=out_dtype,
                                    output_final_state=False)
    assert state is None
    check_forward(x, out, None, "mixed", 1.0)


def side_by_side(x, lens):
    """The packed sequences [N, longest, ...]; behind a sequence's end there are no keys, no decays, nothing."""
    at = torch.arange(max(lens))
    real = at < torch.tensor(lens)[:, None]
    index = (torch.tensor([0] + lens[:-1]).cumsum(0)[:, None] + at).clamp(max=sum(lens) - 1)
    y = {n: t[index.cuda()] for n, t in x.items() if n in ("q", "k", "v", "log_alpha", "d_out")}
    for t in y.values():
        t[~real.cuda()] = 0
    for n in ("state", "d_final"):
        if n in x:
            y[n] = x[n]
    return y, real.cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("longest,count", [(5, 61), (40, 300), (130, 100)])
def test_many_short_sequences(longest, count, d):
    g = torch.Generator().manual_seed(75)
    lens = torch.randint(0, longest + 1, (count,), generator=g).tolist()
    lens[3], lens[7] = longest, 0
    x = with_gradients(lens, 2, d, "mixed", 76)
    y, real = side_by_side(x, lens)
    ref, last = forward(*(y[n] for n in ("q", "k", "v", "log_alpha", "state")))
    a = absolute(y)
    m, ml = forward(*(a[n] for n in ("q", "k", "v", "log_alpha", "state")))
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], cu_seqlens=x["cu"])
    close(out, ref[real], m[real], FINE, 2.0 ** -24, "out")
    close(state, last, ml, FINE, 2.0 ** -24, "state")
    got = gradients(x)
    padded = {}
    for n in ("q", "k", "v", "log_alpha"):
        padded[n] = torch.zeros_like(y[n])
        padded[n][real] = got[n]
    ref, mass = backward(**y), backward(**a)
    for n in ("q", "k", "v", "log_alpha"):  # of tokens that there are
        for t in (ref, mass):
            t[n] = torch.where(real.view(*real.shape, *[1] * (t[n].dim() - 2)), t[n], 0)
        near = mass[n].unflatten(1, (1, -1)).amax(2) if n == "log_alpha" and longest <= 128 else mass[n].amax(1, keepdim=True)
        steps = 2.0 ** -7 + FINE if n == "log_alpha" else 2.0 ** -8 + FINE
        close(padded[n], ref[n], mass[n] + (2.0 ** -17 / steps * near if n == "log_alpha" else 0), steps, 2.0 ** -8, n)
    close(got["initial_state"], ref["initial_state"], mass["initial_state"], FINE, 2.0 ** -24, "initial_state")
    assert kda.kda_last_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 77, 128, 299])
def test_a_value_that_is_not_finite_stays_in_its_channel(at, what, last, out_dtype, d):
    x = on_gpu(inputs((1, 300), 2, d, "slow", 77))
    call = lambda: kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], out_dtype=out_dtype, output_final_state=last)  # noqa: E731
    clean, _ = call()
    x["v"][:, at, 1, 5] = what
    dirty, state = call()
    others = torch.arange(d) != 5
    assert torch.equal(clean[:, :at], dirty[:, :at]) and torch.equal(clean[:, :, 0], dirty[:, :, 0])
    assert torch.equal(clean[..., others], dirty[..., others])
    assert not torch.isfinite(dirty[0, at:, 1, 5]).any()
    if last:
        assert not torch.isfinite(state[0, 1, :, 5]).any() and torch.isfinite(state[0, 0]).all()


@pytest.mark.parametrize("tensor", ["q", "k"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [5, 127, 128, 260])
def test_a_query_or_key_that_is_not_finite_is_not_seen_before(at, out_dtype, d, tensor):
    x = on_gpu(inputs((1, 300), 2, d, "slow", 78))
    clean, _ = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], out_dtype=out_dtype)
    x[tensor][:, at, 1, 5] = float("nan")
    dirty, _ = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], out_dtype=out_dtype)
    assert torch.equal(clean[:, :at], dirty[:, :at]) and torch.equal(clean[:, :, 0], dirty[:, :, 0])
    assert not torch.isfinite(dirty[0, at, 1]).any()
    if tensor == "q":
        assert torch.equal(clean[:, at + 1:], dirty[:, at + 1:])
    else:
        assert not torch.isfinite(dirty[0, at:, 1]).any()
