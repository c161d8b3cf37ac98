"""Gradients of the linear attention where inputs hold values that are not finite: what the formulas put them into is not
finite, and everything else is as close to the formulas as without them (the bounds of test_linear_cuts_gpu.py)."""
import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from linear_cases import absolute, backward, close, inputs
from test_linear_gpu import FINE, on_gpu

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def check(where, d, kind="slow", T=300):
    """where: (tensor, token, channel, value) of head 1."""
    x = on_gpu(inputs((1, T), 2, d, kind, 81, ("q", "k", "v", "d_out")))
    x["state"], x["d_final"] = (torch.randn((1, 2, d, d), device="cuda") for _ in range(2))
    call = lambda: kda.kda_linear_bwd(x["q"], x["k"], x["v"], x["log_alpha"], x["d_out"], initial_state=x["state"],  # noqa: E731
                                      d_final_state=x["d_final"])
    clean = call()
    for n, t, c, _ in where:
        x[n][0, t, 1, c] = 0
    mass = backward(**absolute(x))
    for n, t, c, value in where:
        x[n][0, t, 1, c] = value
    ref, got = backward(**x), call()
    for n in ("q", "k", "v", "log_alpha", "initial_state"):
        assert torch.equal(clean[n][:, :, 0] if n != "initial_state" else clean[n][:, 0],
                           got[n][:, :, 0] if n != "initial_state" else got[n][:, 0]), n
        fin = torch.isfinite(ref[n])
        assert fin.any() or n == "log_alpha"
        assert not torch.isfinite(got[n][~fin]).any(), n
        m, steps, half = mass[n], 2.0 ** -8 + FINE, 2.0 ** -8
        if n == "log_alpha":
            steps = 2.0 ** -7 + FINE
            near = torch.nn.functional.pad(m, (0, 0, 0, -T % 128)).unflatten(1, (-1, 128)).amax(2, keepdim=True)
            m = m + 2.0 ** -17 / steps * near.expand(-1, -1, 128, -1).flatten(1, 2)[:, :T]
        if n == "initial_state":
            steps, half = FINE, 2.0 ** -24
        close(got[n][fin], ref[n][fin], m[fin], steps, half, n)
    assert kda.kda_last_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tensor", ["q", "k", "v", "d_out"])
@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("at", [0, 77, 127, 128, 200, 299])
def test_one(at, what, tensor, d):
    check([(tensor, at, 5, what)], d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", [
    [("q", 10, 3, NAN), ("k", 100, 4, INF)], [("d_out", 140, 0, INF), ("v", 201, 63, NAN)],
    [("q", 130, 60, NAN), ("q", 250, 60, INF), ("k", 131, 60, NAN)], [("k", t, t % 64, NAN) for t in range(40, 90)],
    [("d_out", 60, 9, NAN), ("d_out", 61, 10, NAN), ("v", 62, 9, NAN)], [("k", 128, 0, NAN), ("k", 127, 63, NAN)]])
def test_several(where, d):
    check(where, d)


@pytest.mark.parametrize("kind", ["mixed", "fast"])
@pytest.mark.parametrize("tensor", ["q", "k", "v", "d_out"])
def test_beside_strong_decays(tensor, kind):
    check([(tensor, 90, 7, NAN)], 128, kind)


@pytest.mark.parametrize("tensor", ["q", "k", "v", "d_out"])
def test_the_sum_of_fixed_decays_gradients(tensor):
    x = on_gpu(inputs((2, 200), 3, 64, "slow", 82, ("q", "k", "v", "d_out")))
    decays = torch.tensor([-0.1, -0.2, -0.3], device="cuda")
    call = lambda: kda.kda_linear_bwd(x["q"], x["k"], x["v"], decays, x["d_out"])["log_alpha"]  # noqa: E731
    clean = call()
    x[tensor][1, 100, 2, 9] = NAN
    dirty = call()
    assert torch.equal(clean[:2], dirty[:2]) and torch.isnan(dirty[2])


def test_packed_neighbours_in_one_tile():
    """Short sequences share a tile of rows: the one with such values is its own matter."""
    lens = [60, 3, 50, 40]
    x = on_gpu(inputs((sum(lens),), 2, 64, "slow", 83, ("q", "k", "v", "d_out")))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    call = lambda: kda.kda_linear_bwd(x["q"], x["k"], x["v"], x["log_alpha"], x["d_out"], cu_seqlens=cu)  # noqa: E731
    clean = call()
    for n in ("q", "k", "v", "d_out"):
        x[n][70, :, 3] = INF
    dirty = call()
    others = torch.ones(sum(lens), dtype=torch.bool)
    others[63:113] = False
    for n in ("q", "k", "v", "log_alpha"):
        assert torch.equal(clean[n][others], dirty[n][others]), n
    assert torch.isfinite(dirty["q"][63:70]).all() and torch.isfinite(dirty["k"][71:113]).all()
    assert torch.isfinite(dirty["v"][71:113]).all() and not torch.isfinite(dirty["log_alpha"][63:113]).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", [[("q", 1500, 3, NAN)], [("k", 1300, 4, INF)], [("d_out", 511, 5, NAN), ("v", 1700, 6, NAN)]])
def test_through_segments(where, d):
    check(where, d, T=2500)
