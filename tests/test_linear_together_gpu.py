"""The linear attention's and the logits' calls as they are used together: packed prompts, speculative steps
from their states, and a training step; and the example's stack with such layers."""
import importlib.util
import os

import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from linear_attention_recurrence_fwd_gb300 import binding
from linear_cases import absolute, backward, close, forward, inputs
from test_linear_gpu import FINE, on_gpu, packed_case
from test_logits_gpu import check, reference, rules

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_prompts_then_drafts_then_steps():
    """Three requests: prompts packed, 4 drafts verified with the logits' rules, accepted, committed; the states then
    equal those of the same tokens all at once, up to the roundings of two-piece operands and of fp32 sums."""
    lens, H, d, K, V = [150, 1, 400], 2, 128, 5, 3000
    N = len(lens)
    x = packed_case(lens, H, d, "mixed", 51)
    start = x["state"].clone()
    _, states = kda.kda_linear_fwd(x["q"], x["k"], x["v"], x["log_alpha"], initial_state=x["state"], cu_seqlens=x["cu"])
    g = torch.Generator().manual_seed(52)
    head = (torch.randn((H * d, V), generator=g) / (H * d) ** 0.5).cuda()
    taken = [[] for _ in range(N)]
    for step in range(3):
        y = on_gpu(inputs((N, K), H, d, "mixed", 60 + step))
        out = kda.kda_linear_verify(y["q"], y["k"], y["v"], y["log_alpha"], states)
        logits = out.flatten(2) @ head
        u = rules(N, K, V, 40, 5, True, 70 + step)
        probs = check(logits, u)
        drafts = probs[:, :K - 1].argmax(-1).to(torch.int32)  # likely ones, so that some are kept
        counts, tokens = kda.kda_draft_accept(drafts, None, probs, torch.rand((N, K), generator=g).cuda())
        kda.kda_linear_commit(y["k"], y["v"], y["log_alpha"], states, counts)
        for n in range(N):
            c = int(counts[n])
            assert 1 <= c <= K and (tokens[n, :c] >= 0).all() and (tokens[n, c:] == -1).all()
            taken[n].append({m: t[n, :c] for m, t in y.items()})
    for n in range(N):
        a = sum(lens[:n])
        whole = {m: torch.cat([x[m][a:a + lens[n]]] + [t[m] for t in taken[n]])[None] for m in ("q", "k", "v", "log_alpha")}
        _, last = forward(whole["q"], whole["k"], whole["v"], whole["log_alpha"], start[n:n + 1])
        m = absolute(whole)
        _, mass = forward(m["q"], m["k"], m["v"], m["log_alpha"], start[n:n + 1].abs())
        close(states[n:n + 1], last, mass, FINE, 2.0 ** -24, f"request {n}")
    assert kda.kda_last_device_status() == 0


def test_a_training_step():
    """out = linear attention, loss = <out, w>: the gradients that autograd needs, from the library's two calls."""
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, log_alpha, state):
            out, last = kda.kda_linear_fwd(q, k, v, log_alpha, initial_state=state, out_dtype=torch.bfloat16)
            ctx.save_for_backward(q, k, v, log_alpha, state)
            return out, last

        @staticmethod
        def backward(ctx, d_out, d_last):
            g = kda.kda_linear_bwd(*ctx.saved_tensors[:4], d_out.contiguous(), initial_state=ctx.saved_tensors[4],
                                   d_final_state=d_last.contiguous())
            return g["q"], g["k"], g["v"], g["log_alpha"], g["initial_state"]

    x = on_gpu(inputs((2, 260), 3, 64, "mixed", 53, ("q", "k", "v", "d_out")))
    x["state"], x["d_final"] = torch.randn((2, 3, 64, 64), device="cuda"), torch.randn((2, 3, 64, 64), device="cuda")
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "log_alpha", "state")]
    out, last = Linear.apply(*leaves)
    torch.autograd.backward([out, last], [x["d_out"], x["d_final"]])
    ref, mass = backward(**x), backward(**absolute(x))
    for leaf, n in zip(leaves, ("q", "k", "v", "log_alpha", "initial_state")):
        m = mass[n]
        if n == "log_alpha":  # see test_linear_bwd_gpu.py
            m = m + 2.0 ** -17 / (2.0 ** -7 + FINE) * m.amax(1, keepdim=True)
        steps = {"log_alpha": 2.0 ** -7 + FINE, "initial_state": FINE}.get(n, 2.0 ** -8 + FINE)
        close(leaf.grad, ref[n], m, steps, 2.0 ** -24 if n == "initial_state" else 2.0 ** -8, n)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("layers", ["lll", "rla"])
def test_speculative_steps_equal_token_by_token(example, layers):
    """As test_hybrid_example_gpu.py, with the same bounds: 2^-5 in total variation covers a few bf16 half-steps a layer."""
    N, K, steps = 4, 3, 5
    rule = dict(temperature=0.9, repetition=1.2)
    fast = example.HybridStack(N, layers, max_tokens=64, seed=3, **rule)
    gen = torch.Generator(device="cuda").manual_seed(7)
    first = torch.arange(N, device="cuda", dtype=torch.int32)
    last, history = first, [[int(t)] for t in first]
    for _ in range(steps):
        counts, tokens, last = fast.step(last, K, gen)
        for n in range(N):
            history[n] += tokens[n, :int(counts[n])].tolist()
    assert fast.lens.tolist() == [len(h) - 1 for h in history]
    for n in range(N):
        assert fast.said[n, :len(history[n])].tolist() == history[n]
    probs = fast.forward(last[:, None])[0][:, 0]
    for n in range(N):
        slow = example.HybridStack(N, layers, max_tokens=64, seed=3, **rule)
        one = torch.ones(N, dtype=torch.int32, device="cuda")
        for t in history[n]:
            p, parts = slow.forward(torch.full((N, 1), t, dtype=torch.int32, device="cuda"))
            if slow.lens[n] < len(history[n]) - 1:
                slow.commit(parts, one)
        assert float((p[n, 0] - probs[n]).abs().sum()) / 2 < 2 ** -5
        for a, b in zip(fast.held, slow.held):
            if isinstance(a, torch.Tensor):
                assert float((a[n] - b[n]).norm() / b[n].norm()) < 2 ** -5
    assert binding.kda_last_device_status() == 0


def test_the_example_runs_with_the_rules(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["hybrid_decode.py", "--requests", "3", "--steps", "4", "--layers", "rlla", "--temperature", "0.8",
                                     "--repetition", "1.1"])
    example.main()
    assert "device status 0" in capsys.readouterr().out


def test_a_repeated_token_is_penalised(example):
    stack = example.HybridStack(1, "l", vocabulary=50, max_tokens=32, seed=5, repetition=4.0)
    token = torch.tensor([[7]], dtype=torch.int32, device="cuda")
    stack.lens.fill_(2)
    stack.said[0, :2] = torch.tensor([9, 11], device="cuda")
    with_, _ = stack.forward(token)
    stack.rules["repetition"].fill_(1.0)
    without, _ = stack.forward(token)
    ref, _ = reference(torch.log(without).cpu(), {})
    assert torch.allclose(without.cpu().double(), ref, atol=1e-5)
    logit_up = without[0, 0, [7, 9, 11]] > with_[0, 0, [7, 9, 11]]
    assert logit_up.any()
    others = torch.ones(50, dtype=torch.bool)
    others[[7, 9, 11]] = False
    ratio = (with_ / without)[0, 0, others]
    assert torch.allclose(ratio, ratio[:1].expand_as(ratio), rtol=1e-4)


def test_offsets_past_32_bits():
    T, cut, H, d = 600_000, 590_000, 32, 128  # 2.5 * 10^9 elements a tensor
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn((1, T, H, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    la = -0.1 * torch.rand((1, T, H), generator=g, device="cuda")
    out, state = kda.kda_linear_fwd(q, k, v, la, scale=d ** -1.0, out_dtype=torch.bfloat16)
    _, before = kda.kda_linear_fwd(q[:, :cut], k[:, :cut], v[:, :cut], la[:, :cut], scale=d ** -1.0, out_dtype=torch.bfloat16)
    tail = [t[:, cut:] for t in (q, k, v, la)]
    out_tail, state_tail = kda.kda_linear_fwd(*tail, before, scale=d ** -1.0, out_dtype=torch.bfloat16)

    def off(a, b):
        return float((a.double() - b.double()).norm() / b.double().norm())

    # both are within 2.5 half-steps of bf16 (fp32 sums of 16-bit numbers for the state) of the same numbers, in the 2-norm
    assert off(out[:, cut:], out_tail) < 2 * 2.5 * 2.0 ** -8 and off(state, state_tail) < 2 * 2.0 ** -15
    a = kda.kda_linear_bwd(q, k, v, la, do, scale=d ** -1.0)
    b = kda.kda_linear_bwd(*tail, do[:, cut:], before, scale=d ** -1.0)
    for n in ("q", "k", "v", "log_alpha"):
        assert off(a[n][:, cut:], b[n]) < 2 * 2.5 * 2.0 ** -8, n


def test_probabilities_past_32_bits():
    N, R, V = 1400, 4, 400_001
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((N, R, V), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    u = {"tokens": torch.randint(0, V, (N, 300), generator=g, device="cuda", dtype=torch.int32),
         "repetition": torch.full((N,), 1.2, device="cuda"),
         "mask": torch.randint(-2 ** 31, 2 ** 31 - 1, (N, R, (V + 31) // 32), generator=g, device="cuda", dtype=torch.int32)}
    p = kda.kda_logits_probs(x, out_dtype=torch.bfloat16, **u)
    last = kda.kda_logits_probs(x[-2:].clone(), out_dtype=torch.bfloat16, **{n: t[-2:].clone() for n, t in u.items()})
    assert torch.equal(p[-2:], last)
