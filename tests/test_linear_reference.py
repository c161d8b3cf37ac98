"""The plain 64-bit forms that the linear attention is tested against, themselves checked: the backward form
against differences and against automatic differentiation, the forward one against the sum over pairs."""
import pytest
import torch

from linear_cases import absolute, backward, forward, inputs


def case(kind, seed, B=2, T=9, H=2, d=4):
    x = inputs((B, T), H, d, kind, seed, ("q", "k", "v", "d_out"))
    g = torch.Generator().manual_seed(seed + 1)
    x = {n: t.double() for n, t in x.items()}
    x["state"], x["d_final"] = (torch.randn((B, H, d, d), generator=g, dtype=torch.float64) for _ in range(2))
    return x


def value(x, scale):
    out, last = forward(x["q"], x["k"], x["v"], x["log_alpha"], x["state"], scale)
    return (out * x["d_out"]).sum() + (last * x["d_final"]).sum()


@pytest.mark.parametrize("kind", ["mixed", "slow", "fast", "none"])
def test_backward_against_differences(kind):
    x = case(kind, 3)
    g = backward(**x, scale=0.7)
    step = 1e-6
    for n in ("q", "k", "v", "log_alpha", "initial_state"):
        name = "state" if n == "initial_state" else n
        at = torch.Generator().manual_seed(5)
        for _ in range(6):
            i = int(torch.randint(x[name].numel(), (1,), generator=at))
            up, down = dict(x), dict(x)
            for y, s in ((up, step), (down, -step)):
                y[name] = x[name].clone()
                y[name].view(-1)[i] += s
            slope = (value(up, 0.7) - value(down, 0.7)) / (2 * step)
            assert abs(slope - g[n].reshape(-1)[i]) < 1e-7 * (1 + abs(slope)), (n, i)


@pytest.mark.parametrize("kind", ["mixed", "reset"])
def test_backward_against_autograd(kind):
    x = case(kind, 4)
    leaves = {n: t.clone().requires_grad_() for n, t in x.items() if n not in ("d_out", "d_final")}
    S, total = leaves["state"], 0
    a = torch.exp(leaves["log_alpha"])
    for t in range(x["q"].shape[1]):
        S = a[:, t, :, None, None] * S + torch.einsum("bhk,bhv->bhkv", leaves["k"][:, t], leaves["v"][:, t])
        total = total + (torch.einsum("bhk,bhkv->bhv", leaves["q"][:, t], S) * x["d_out"][:, t]).sum()
    (total + (S * x["d_final"]).sum()).backward()
    g = backward(**x)
    for n, t in leaves.items():
        m = "initial_state" if n == "state" else n
        assert torch.allclose(g[m], t.grad, rtol=1e-10, atol=1e-12), n


def test_forward_is_the_sum_over_pairs():
    x = case("mixed", 6)
    out, _ = forward(x["q"], x["k"], x["v"], x["log_alpha"], None)
    G = x["log_alpha"].cumsum(1)
    w = torch.einsum("bihd,bjhd->bhij", x["q"], x["k"]) * torch.exp((G[:, :, None] - G[:, None]).permute(0, 3, 1, 2)).tril()
    assert torch.allclose(out, torch.einsum("bhij,bjhd->bihd", w, x["v"]), rtol=1e-10, atol=1e-12)


def test_a_planted_mistake_is_seen():
    x = case("mixed", 7)
    g = backward(**x)
    late = dict(x, log_alpha=x["log_alpha"].roll(1, 1))  # each decay one token too late
    mass = backward(**absolute(x))
    for n in ("q", "k", "v", "log_alpha", "initial_state"):
        assert ((g[n] - backward(**late)[n]).abs() > 2.0 ** -6 * mass[n]).any(), n
