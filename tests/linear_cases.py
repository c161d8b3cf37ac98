"""Inputs and plain 64-bit forms of the linear attention with one decay per head.

Every tolerance is a number of half-steps of a type times the `mass` of a result: the same sums with every
factor replaced by its absolute value, which bounds what a relative error of each factor can do."""
import torch

KINDS = ("mixed", "slow", "fast", "none", "reset")


def decays(kind, shape, g):
    """log_alpha of one kind: fp32 numbers that bf16 holds."""
    n = torch.randn(shape, generator=g)
    x = {"mixed": -torch.exp(2 * n - 3), "slow": -1e-3 * torch.exp(n), "fast": -8 * torch.rand(shape, generator=g),
         "none": torch.zeros(shape), "reset": -0.05 * torch.rand(shape, generator=g)}[kind]
    if kind == "reset":
        x[torch.rand(shape, generator=g) < 0.04] = -float("inf")
    return x.to(torch.bfloat16)


def inputs(lead, H, d, kind="mixed", seed=0, names=("q", "k", "v")):
    """bf16 tensors [*lead, H, d] of unit variance (q and k over sqrt(d)) and log_alpha [*lead, H]."""
    g = torch.Generator().manual_seed(seed)
    got = {}
    for n in names:
        x = torch.randn((*lead, H, d), generator=g)
        got[n] = (x / d ** 0.5 if n in ("q", "k") else x).to(torch.bfloat16)
    got["log_alpha"] = decays(kind, (*lead, H), g)
    return got


def forward(q, k, v, log_alpha, state, scale=1.0):
    """Token after token in 64 bits; q, k, v [B, T, H, d], log_alpha [B, T, H], state [B, H, d, d] or None.
    Returns (out, final state)."""
    q, k, v, a = q.double(), k.double(), v.double(), torch.exp(log_alpha.double())
    B, T, H, d = q.shape
    S = torch.zeros((B, H, d, d), dtype=torch.float64, device=q.device) if state is None else state.double().clone()
    out = torch.zeros_like(q)
    for t in range(T):
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        out[:, t] = scale * torch.matmul(q[:, t, :, None], S)[:, :, 0]
    return out, S


def backward(q, k, v, log_alpha, d_out, state, d_final, scale=1.0):
    """The same recurrence backwards: gradients of <d_out, out> + <d_final, final state>."""
    q, k, v, a, do = q.double(), k.double(), v.double(), torch.exp(log_alpha.double()), scale * d_out.double()
    B, T, H, d = q.shape
    zero = torch.zeros((B, H, d, d), dtype=torch.float64, device=q.device)
    states = [zero if state is None else state.double()]
    for t in range(T):
        states.append(a[:, t, :, None, None] * states[-1] + k[:, t, :, :, None] * v[:, t, :, None, :])
    G = zero if d_final is None else d_final.double()
    g = {"q": torch.zeros_like(q), "k": torch.zeros_like(q), "v": torch.zeros_like(q), "log_alpha": torch.zeros_like(a)}
    for t in range(T - 1, -1, -1):
        g["q"][:, t] = torch.matmul(states[t + 1], do[:, t, :, :, None])[..., 0]
        G = G + q[:, t, :, :, None] * do[:, t, :, None, :]
        g["k"][:, t] = torch.matmul(G, v[:, t, :, :, None])[..., 0]
        g["v"][:, t] = torch.matmul(k[:, t, :, None], G)[:, :, 0]
        G = a[:, t, :, None, None] * G
        g["log_alpha"][:, t] = (G * states[t]).sum((-1, -2))
    g["initial_state"] = G
    return g


def absolute(x):
    """The arguments' absolute values (log_alpha as it is)."""
    return {n: t if n == "log_alpha" or t is None else t.double().abs() for n, t in x.items()}


def close(got, ref, mass, steps, half, name=""):
    """|got - ref| <= half |ref| + steps mass, everywhere; exact zeros of the mass are exact zeros."""
    if not got.numel():
        return
    got, ref = got.double().cpu(), ref.double().cpu()
    bound = half * ref.abs() + steps * mass.double().cpu() + 1e-30
    over = (got - ref).abs() / bound
    assert torch.isfinite(got).all(), name
    assert over.max() <= 1, f"{name}: {over.max():.3g} times the bound at {int(over.argmax())}"
