"""kda_linear_bwd against the recurrence backwards in 64 bits.

Bounds.  A gradient is a sum of products of inputs, of weights (one rounding to bf16, 2^-8) and of states and
their gradients (one rounding to bf16 as an operand, and two-piece operands where they are formed), and is
rounded to its type at the end: 2^-8 of the mass for either operand's rounding, 2^-14 of it for fp32 sums,
decays and two-piece operands (2^-11 with resets), and the type's own half-step.  The initial state's
gradient is formed of two-piece operands alone.
A decay's gradient D_t is a sum over the pairs of tokens on either side of t.  Neighbours differ by what token t
takes out and brings in, so within a chunk of 128 tokens it is a running sum of differences: 128 fp32 roundings
of partial sums, each at most the largest D's mass in the chunk, 128 * 2^-24 = 2^-17 of that largest mass, which
is all that is left where D itself is 0 (a first token without a state before it, a reset)."""
import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from linear_cases import KINDS, absolute, backward, close, inputs
from test_linear_gpu import FINE, RESET, half, on_gpu

pytestmark = pytest.mark.gpu


def check(x, g, kind, scale=1.0, la_dtype=torch.bfloat16):
    keys = ("q", "k", "v", "log_alpha", "d_out", "state", "d_final")
    x = {n: x.get(n) for n in keys}
    ref, mass = backward(**x, scale=scale), backward(**absolute(x), scale=abs(scale))
    fine = RESET if kind == "reset" else FINE
    for n in ("q", "k", "v"):
        assert g[n].dtype == torch.bfloat16
        close(g[n], ref[n], mass[n], 2.0 ** -8 + fine, 2.0 ** -8, n)
    if g["log_alpha"] is not None:
        assert g["log_alpha"].dtype == la_dtype
        m = mass["log_alpha"] + 2.0 ** -17 / (2.0 ** -7 + fine) * mass["log_alpha"].amax(1, keepdim=True)
        close(g["log_alpha"], ref["log_alpha"], m, 2.0 ** -7 + fine, half(la_dtype), "log_alpha")
    if g["initial_state"] is not None:
        close(g["initial_state"], ref["initial_state"], mass["initial_state"], fine, 2.0 ** -24, "initial_state")


def case(lead, N, H, d, kind, seed, start=True):
    x = on_gpu(inputs(lead, H, d, kind, seed, ("q", "k", "v", "d_out")))
    x["state"], x["d_final"] = (torch.randn((N, H, d, d), device="cuda") if start else None for _ in range(2))
    return x


def run(x, **kw):
    return kda.kda_linear_bwd(x["q"], x["k"], x["v"], x["log_alpha"], x["d_out"], initial_state=x["state"],
                              d_final_state=x["d_final"], **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,T,H,start", [(1, 1, 1, True), (2, 7, 3, False), (1, 128, 2, True), (3, 129, 1, True),
                                         (1, 300, 5, False), (2, 513, 2, True)])
def test_fixed_lengths(B, T, H, start, kind, d):
    x = case((B, T), B, H, d, kind, T, start)
    check(x, run(x, scale=0.6), kind, 0.6)
    assert kda.kda_last_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[5], [1, 0, 128, 3], [130, 1, 255, 0, 64, 300], [0, 0, 7]])
def test_packed(lens, d):
    x = case((sum(lens),), len(lens), 2, d, "mixed", 31)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    g = run(x, cu_seqlens=cu)
    a = 0
    for n, L in enumerate(lens):
        y = {m: x[m][a:a + L][None] for m in ("q", "k", "v", "log_alpha", "d_out")}
        y["state"], y["d_final"] = x["state"][n:n + 1], x["d_final"][n:n + 1]
        part = {m: g[m][a:a + L][None] for m in ("q", "k", "v", "log_alpha")}
        part["initial_state"] = g["initial_state"][n:n + 1]
        if L:
            check(y, part, "mixed")
        else:
            assert torch.equal(part["initial_state"], y["d_final"])
        a += L
    assert kda.kda_last_device_status() == 0


@pytest.mark.parametrize("B,T,H,d", [(1, 5000, 2, 128), (2, 1700, 1, 64)])
def test_long(B, T, H, d):
    x = case((B, T), B, H, d, "slow", 32)
    check(x, run(x), "slow")


def test_sequences_do_not_reach_one_another():
    lens = [70, 200, 5, 131]
    x = case((sum(lens),), 4, 2, 128, "mixed", 33)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    clean = run(x, cu_seqlens=cu)
    for n in ("q", "k", "v", "log_alpha", "d_out"):
        x[n][70:270] = float("nan")
    x["state"][1] = x["d_final"][1] = float("nan")
    dirty = run(x, cu_seqlens=cu)
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[70:270] = False
    for n in ("q", "k", "v", "log_alpha"):
        assert torch.equal(clean[n][keep], dirty[n][keep]), n
    others = [0, 2, 3]
    assert torch.equal(clean["initial_state"][others], dirty["initial_state"][others])


def test_fixed_decays_get_the_sum():
    B, T, H, d = 2, 333, 3, 64
    x = case((B, T), B, H, d, "mixed", 34)
    fixed = -torch.tensor([0.0, 0.02, 0.9], device="cuda")
    x["log_alpha"] = fixed
    g = run(x)
    assert g["log_alpha"].shape == (H,) and g["log_alpha"].dtype == torch.float32
    x["log_alpha"] = fixed.expand(B, T, H)
    by_token = run(x)
    assert by_token["log_alpha"].shape == (B, T, H)
    for n in ("q", "k", "v", "initial_state"):
        assert torch.equal(g[n], by_token[n])
    y = {n: x.get(n) for n in ("q", "k", "v", "log_alpha", "d_out", "state", "d_final")}
    ref, mass = backward(**y), backward(**absolute(y))
    close(g["log_alpha"], ref["log_alpha"].sum((0, 1)), mass["log_alpha"].sum((0, 1)), 2.0 ** -8 + FINE, 2.0 ** -24, "sum")
    check(x, by_token, "mixed", la_dtype=torch.float32)


def test_slices_and_what_is_left_out():
    B, T, H, d = 2, 140, 2, 128
    x = case((B, T), B, H, d, "mixed", 35)
    want = run(x)
    side = torch.cat([x["q"], x["k"], x["v"], x["d_out"]], 2)
    y = dict(x)
    y["q"], y["k"], y["v"], y["d_out"] = side.split(H, dim=2)
    got = run(y)
    for n in want:
        assert torch.equal(want[n], got[n]), n
    got = run(y, want_log_alpha_grad=False, want_initial_state_grad=False)
    assert got["log_alpha"] is None and got["initial_state"] is None
    for n in ("q", "k", "v"):
        assert torch.equal(want[n], got[n]), n


def test_repeats_streams_and_graphs():
    x = case((1, 600), 1, 2, 128, "mixed", 36)
    want = run(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    again = run(x, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(x)
    graph.replay()
    for n in want:
        assert torch.equal(want[n], again[n]) and torch.equal(want[n], held[n]), n


def test_against_differences_of_the_forward_call():
    """Along one direction of every input: the forward call's own values, in fp32, at steps wide enough for
    bf16 inputs (powers of two times a sign, so that inputs and differences are exact)."""
    x = case((1, 200), 1, 2, 64, "slow", 37)
    g = run(x)
    for n in ("q", "k", "v"):
        direction = torch.sign(torch.randn_like(x[n].float()))
        step = 2.0 ** -4
        ends = []
        for s in (step, -step):
            y = dict(x)
            y[n] = (x[n].float() + s * direction).to(torch.bfloat16)
            out, last = kda.kda_linear_fwd(y["q"], y["k"], y["v"], y["log_alpha"], initial_state=x["state"])
            # the operator is linear in each of q, k and v: only the inputs' rounding is left to account for
            ends.append(((out.double() * x["d_out"].double()).sum() + (last.double() * x["d_final"].double()).sum(), y[n]))
        moved = ends[0][1].double() - ends[1][1].double()
        slope = (g[n].double() * moved).sum()
        noise = (g[n].double() * moved).norm()  # gradients are rounded to bf16, independently
        assert abs(ends[0][0] - ends[1][0] - slope) <= 4 * 2.0 ** -7 * noise + 2.0 ** -12 * abs(slope), n


def test_empty():
    z = torch.empty((2, 0, 3, 64), dtype=torch.bfloat16, device="cuda")
    ds = torch.randn((2, 3, 64, 64), device="cuda")
    g = kda.kda_linear_bwd(z, z, z, z[..., 0], z, d_final_state=ds)
    assert torch.equal(g["initial_state"], ds) and g["q"].shape == z.shape
    g = kda.kda_linear_bwd(z, z, z, torch.zeros(3, device="cuda"), z)
    assert (g["initial_state"] == 0).all() and (g["log_alpha"] == 0).all()
