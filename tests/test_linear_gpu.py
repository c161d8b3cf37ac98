"""The linear attention's forward calls against the recurrence in 64 bits.

Bounds.  Every operand of a product that is not an input is rounded: to two bf16 numbers (16 bits: 2^-16), or
with 16-bit outputs, weights and states that only outputs see, to one (2^-8); a result's own rounding comes on
top.  Sums, decays and exponentials are fp32: 2^-14 of the mass covers them and two-piece operands with room
for the sums' lengths here.  (A decay is off by 2^-24 of the running sum of its chunk, a few hundred at most
but for resets, which add 150 each: under 2^-11 for the 20 that a chunk here has at most, see the reset case.)"""
import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from linear_attention_recurrence_fwd_gb300 import binding
from linear_cases import KINDS, absolute, close, forward, inputs

pytestmark = pytest.mark.gpu

FINE, RESET = 2.0 ** -14, 2.0 ** -11


def on_gpu(x):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}


def steps(kind, out_dtype=torch.float32):
    return (RESET if kind == "reset" else FINE) + (2 * 2.0 ** -8 if out_dtype == torch.bfloat16 else 0)


def half(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def check_forward(x, out, state, kind, scale, **where):
    ref, last = forward(x["q"], x["k"], x["v"], x["log_alpha"], x.get("state"), scale)
    a = absolute(x)
    m, ml = forward(a["q"], a["k"], a["v"], a["log_alpha"], a.get("state"), abs(scale))
    close(out, ref, m, steps(kind, out.dtype), half(out.dtype), "out")
    if state is not None:
        close(state, last, ml, steps(kind), 2.0 ** -24, "state")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,T,H,start", [(1, 1, 1, True), (2, 7, 3, False), (1, 128, 2, True), (3, 129, 1, True),
                                         (1, 300, 5, False), (2, 513, 2, True)])
def test_fixed_lengths(B, T, H, start, kind, out_dtype, d):
    x = on_gpu(inputs((B, T), H, d, kind, seed=T + H))
    x["state"] = torch.randn((B, H, d, d), device="cuda") if start else None
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], scale=0.6,
                                    out_dtype=out_dtype)
    assert out.dtype == out_dtype
    check_forward(x, out, state, kind, 0.6)
    assert kda.kda_last_device_status() == 0


def packed_case(lens, H, d, kind, seed, rows_after=0):
    T = sum(lens) + rows_after
    x = on_gpu(inputs((T,), H, d, kind, seed))
    x["cu"] = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    x["state"] = torch.randn((len(lens), H, d, d), device="cuda")
    return x


def sequence(x, n, lens):
    a = sum(lens[:n])
    y = {m: x[m][a:a + lens[n]][None] for m in ("q", "k", "v", "log_alpha")}
    y["state"] = x["state"][n:n + 1]
    return y, slice(a, a + lens[n])


@pytest.mark.parametrize("d,out_dtype", [(64, torch.float32), (128, torch.bfloat16), (128, torch.float32)])
@pytest.mark.parametrize("lens", [[5], [1, 0, 128, 3], [130, 1, 255, 0, 64, 300], [0, 0, 7], [33] * 9])
def test_packed(lens, d, out_dtype):
    x = packed_case(lens, 3, d, "mixed", 11)
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"],
                                    cu_seqlens=x["cu"], out_dtype=out_dtype)
    for n in range(len(lens)):
        y, rows = sequence(x, n, lens)
        check_forward(y, out[rows][None], state[n:n + 1], "mixed", 1.0)
    assert kda.kda_last_device_status() == 0


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_sequences_do_not_reach_one_another(what):
    lens = [70, 200, 5, 131]
    x = packed_case(lens, 2, 128, "mixed", 12)
    clean, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], cu_seqlens=x["cu"])
    for n in ("q", "k", "v"):
        x[n][70:270] = what
    x["log_alpha"][70:270] = float("nan")
    x["state"][1] = what
    dirty, last = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], cu_seqlens=x["cu"])
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[70:270] = False
    assert torch.equal(clean[keep], dirty[keep])
    assert torch.equal(state[[0, 2, 3]], last[[0, 2, 3]])
    assert not torch.isfinite(dirty[70:270]).any()


@pytest.mark.parametrize("tensor", ["q", "k", "v"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 77, 127, 128, 250, 299])
def test_later_tokens_are_not_seen(at, what, tensor):
    x = on_gpu(inputs((1, 300), 2, 128, "slow", 13))
    clean, _ = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"])
    x[tensor][:, at, 1, 5] = what
    dirty, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"])
    assert torch.equal(clean[:, :at], dirty[:, :at]) and torch.equal(clean[:, :, 0], dirty[:, :, 0])
    channel = dirty[0, at:, 1, 5] if tensor == "v" else dirty[0, at, 1]
    assert not torch.isfinite(channel).any()
    if tensor == "v":
        others = torch.arange(128) != 5
        assert torch.equal(clean[..., others], dirty[..., others])
        assert not torch.isfinite(state[0, 1, :, 5]).any()


@pytest.mark.parametrize("d", [64, 128])
def test_slices_of_one_projection_and_fixed_decays(d):
    B, T, H = 2, 150, 3
    x = on_gpu(inputs((B, T), H, d, "mixed", 14))
    side = torch.cat([x["q"], x["k"], x["v"]], 2)
    q, k, v = side.split(H, dim=2)
    fixed = -torch.tensor([0.0, 0.01, 0.7], device="cuda")
    out, state = kda.kda_linear_fwd(q, k, v, fixed)
    x["log_alpha"], x["state"] = fixed.expand(B, T, H), None
    check_forward(x, out, state, "mixed", 1.0)
    wide = torch.zeros((B, T, 2 * H), device="cuda")
    wide[..., ::2] = fixed
    again, _ = kda.kda_linear_fwd(q, k, v, wide[..., ::2])
    assert torch.equal(out, again)


def test_rows_without_a_sequence_and_bad_offsets():
    x = packed_case([40, 90], 2, 64, "mixed", 15)
    for bad in ([0, 40, 100], [3, 40, 130], [0, 90, 40], [0, 40, 500], [-5, 40, 130]):
        out = torch.full((130, 2, 64), 7.0, device="cuda")
        around = torch.full((132, 2, 64), 7.0, device="cuda")
        around[1:131] = out
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], cu_seqlens=cu, out=around[1:131])
        assert kda.kda_last_device_status() == 1, bad
        assert (around[0] == 7).all() and (around[131] == 7).all()
        if bad == [0, 40, 100]:
            assert (around[101:131] == 7).all()
    cu = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")
    empty = x["q"][:0]
    out, state = kda.kda_linear_fwd(empty, empty, empty, x["log_alpha"][:0], initial_state=x["state"], cu_seqlens=cu)
    assert out.numel() == 0 and torch.equal(state, x["state"])
    assert kda.kda_last_device_status() == 0


def test_empty_batches():
    z = torch.empty((2, 0, 3, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.randn((2, 3, 64, 64), device="cuda")
    out, state = kda.kda_linear_fwd(z, z, z, z[..., 0], initial_state=s)
    assert out.shape == z.shape and torch.equal(state, s)
    _, state = kda.kda_linear_fwd(z, z, z, z[..., 0])
    assert (state == 0).all()
    z = torch.empty((0, 5, 3, 64), dtype=torch.bfloat16, device="cuda")
    out, state = kda.kda_linear_fwd(z, z, z, z[..., 0])
    assert out.shape == z.shape and state.shape == (0, 3, 64, 64)


@pytest.mark.parametrize("B,T,H", [(1, 5000, 2), (2, 2600, 3), (1, 20000, 1)])
@pytest.mark.parametrize("kind", ["slow", "mixed"])
def test_long_prompts_are_cut_and_joined(B, T, H, kind):
    x = on_gpu(inputs((B, T), H, 128, kind, 16))
    x["state"] = torch.randn((B, H, 128, 128), device="cuda")
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"])
    check_forward(x, out, state, kind, 1.0)


def test_long_packed_prompts():
    lens = [1, 4100, 0, 700, 2, 9000, 129]
    x = packed_case(lens, 2, 128, "slow", 17)
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], cu_seqlens=x["cu"],
                                    out_dtype=torch.bfloat16)
    for n in range(len(lens)):
        y, rows = sequence(x, n, lens)
        if lens[n]:
            check_forward(y, out[rows][None], state[n:n + 1], "slow", 1.0)
        else:
            assert torch.equal(state[n], x["state"][n])


def test_state_in_place_split_and_repeat():
    x = on_gpu(inputs((2, 400), 2, 128, "slow", 18))
    s = torch.randn((2, 2, 128, 128), device="cuda")
    whole, last = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=s)
    again, last2 = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=s)
    assert torch.equal(whole, again) and torch.equal(last, last2)
    held = s.clone()
    for part in (slice(0, 256), slice(256, 400)):
        y = {n: t[:, part].contiguous() for n, t in x.items()}
        out, state = kda.kda_linear_fwd(y["q"], y["k"], y["v"], y["log_alpha"], initial_state=held, final_state=held)
        assert state is held
        assert (out - whole[:, part]).abs().max() < 1e-3
    assert (held - last).norm() <= 2.0 ** -15 * last.norm()


def test_long_prompt_with_its_state_in_place():
    x = on_gpu(inputs((2, 6000), 3, 128, "slow", 26))
    s = torch.randn((2, 3, 128, 128), device="cuda")
    want, last = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=s)
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=s, final_state=s)
    assert state is s and torch.equal(out, want) and torch.equal(s, last)


def test_captured_and_replayed_on_another_stream():
    x = on_gpu(inputs((1, 700), 2, 128, "mixed", 19))
    want, last = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], stream=stream)
    stream.synchronize()
    assert torch.equal(out, want) and torch.equal(state, last)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, state = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"])
    for seed in (20, 21):
        for n, t in inputs((1, 700), 2, 128, "mixed", seed).items():
            x[n].copy_(t)
        graph.replay()
        want, last = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"])
        assert torch.equal(out, want) and torch.equal(state, last)


# ---------------------------------------------------------------- tokens

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,H", [(1, 1), (5, 3), (64, 8)])
def test_step(N, H, out_dtype, d):
    x = on_gpu(inputs((N,), H, d, "reset", N))
    s = torch.randn((N, H, d, d), device="cuda")
    held = s.clone()
    out = kda.kda_linear_step(x["q"], x["k"], x["v"], x["log_alpha"], held, scale=0.5, out_dtype=out_dtype)
    y = {n: t[:, None] for n, t in x.items()}
    y["state"] = s
    ref, last = forward(y["q"], y["k"], y["v"], y["log_alpha"], s, 0.5)
    a = absolute(y)
    m, ml = forward(a["q"], a["k"], a["v"], a["log_alpha"], a["state"], 0.5)
    # fp32 throughout: an exponential, a product and a sum; then sums of d terms
    close(held, last, ml, 4 * 2.0 ** -24, 0, "state")
    close(out[:, None], ref, m, (4 + d) * 2.0 ** -24, half(out_dtype), "out")


@pytest.mark.parametrize("d,H", [(64, 3), (128, 2)])
@pytest.mark.parametrize("K", [1, 2, 4, 5, 9, 19])
def test_verify_and_commit(K, d, H):
    N = 7
    x = on_gpu(inputs((N, K), H, d, "mixed", K))
    s = torch.randn((N, H, d, d), device="cuda")
    held = s.clone()
    out = kda.kda_linear_verify(x["q"], x["k"], x["v"], x["log_alpha"], held)
    assert torch.equal(held, s)
    steps_ = s.clone()
    accepted = torch.randint(-1, K + 3, (N,), dtype=torch.int32, device="cuda")
    kept = s.clone()
    for t in range(K):
        one = kda.kda_linear_step(*(x[n][:, t] for n in ("q", "k", "v")), x["log_alpha"][:, t], steps_)
        assert torch.equal(one, out[:, t])
        kept = torch.where((accepted > t)[:, None, None, None], steps_, kept)
    kda.kda_linear_commit(x["k"], x["v"], x["log_alpha"], held, accepted)
    assert torch.equal(held, kept)
    ref, _ = forward(x["q"], x["k"], x["v"], x["log_alpha"], s)
    a = absolute(x)
    m, _ = forward(a["q"], a["k"], a["v"], a["log_alpha"], s.abs())
    close(out, ref, m, (4 * K + 4 + d) * 2.0 ** -24, 2.0 ** -24, "out")


def test_steps_follow_a_prompt():
    x = on_gpu(inputs((2, 140), 3, 64, "mixed", 23))
    want, last = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"])
    y = {n: t[:, :137].contiguous() for n, t in x.items()}
    _, state = kda.kda_linear_fwd(y["q"], y["k"], y["v"], y["log_alpha"])
    for t in range(137, 140):
        out = kda.kda_linear_step(*(x[n][:, t] for n in ("q", "k", "v")), x["log_alpha"][:, t], state)
        assert (out - want[:, t]).abs().max() < 1e-3
    assert (state - last).norm() <= 2.0 ** -15 * last.norm()


def test_step_slices_and_fixed_decays():
    N, H, d = 4, 2, 128
    x = on_gpu(inputs((N,), H, d, "mixed", 24))
    q, k, v = torch.cat([x["q"], x["k"], x["v"]], 1).split(H, dim=1)
    fixed = torch.tensor([-0.5, -0.25], device="cuda")
    a = torch.zeros((N, H, d, d), device="cuda")
    b = a.clone()
    out = kda.kda_linear_step(q, k, v, fixed, a)
    same = kda.kda_linear_step(x["q"], x["k"], x["v"], fixed.expand(N, H).contiguous(), b)
    assert torch.equal(out, same) and torch.equal(a, b)


def test_heads_of_a_single_token_must_be_packed():
    x = on_gpu(inputs((1,), 2, 64, "mixed", 26))
    s = torch.zeros((1, 2, 64, 64), device="cuda")
    apart = {n: torch.cat([x[n], x[n]], -1)[..., :64] for n in "qkv"}  # the same values, heads 128 apart
    for n in "qkv":
        y = {**x, n: apart[n]}
        with pytest.raises(ValueError):
            kda.kda_linear_step(y["q"], y["k"], y["v"], x["log_alpha"], s)
        with pytest.raises(ValueError):
            kda.kda_linear_fwd(y["q"][None], y["k"][None], y["v"][None], x["log_alpha"][None])
    with pytest.raises(ValueError):
        kda.kda_linear_step(*apart.values(), x["log_alpha"], s)
    # a token's own place in a longer row is no matter
    inside = {n: torch.cat([x[n], x[n]], 1)[:, :2] for n in "qkv"}
    a, b = s.clone(), s.clone()
    assert torch.equal(kda.kda_linear_step(x["q"], x["k"], x["v"], x["log_alpha"], a),
                       kda.kda_linear_step(*inside.values(), x["log_alpha"], b)) and torch.equal(a, b)


def test_arguments_are_checked():
    x = on_gpu(inputs((2, 5), 2, 64, "mixed", 25))
    q, k, v, la = x["q"], x["k"], x["v"], x["log_alpha"]
    s = torch.zeros((2, 2, 64, 64), device="cuda")
    for call in (lambda: kda.kda_linear_fwd(q[:, :4], k, v, la), lambda: kda.kda_linear_fwd(q.float(), k, v, la),
                 lambda: kda.kda_linear_fwd(q, k, v, la[:, :4]), lambda: kda.kda_linear_fwd(q, k, v, la.half()),
                 lambda: kda.kda_linear_fwd(q, k, v, la, initial_state=s[:1]),
                 lambda: kda.kda_linear_fwd(q, k, v, la, out_dtype=torch.float16),
                 lambda: kda.kda_linear_fwd(q[0], k[0], v[0], la[0]),
                 lambda: kda.kda_linear_fwd(q.cpu(), k, v, la),
                 lambda: kda.kda_linear_fwd(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), la.transpose(1, 2)),
                 lambda: kda.kda_linear_step(q[:, 0], k[:, 0], v[:, 0], la[:, 0], s[:, :, :32]),
                 lambda: kda.kda_linear_commit(k, v, la, s, torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    wide = inputs((2, 5), 2, 32, "mixed", 25)
    with pytest.raises(binding.KDAError) as e:
        kda.kda_linear_fwd(wide["q"].cuda(), wide["k"].cuda(), wide["v"].cuda(), wide["log_alpha"].cuda())
    assert e.value.code == 2
    odd = torch.zeros((2, 5, 2 * 64 + 1), dtype=torch.bfloat16, device="cuda")[..., 1:].unflatten(-1, (2, 64))
    with pytest.raises(binding.KDAError) as e:
        kda.kda_linear_fwd(odd, k, v, la)
    assert e.value.code == 3
