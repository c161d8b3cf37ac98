"""The example's stack: speculative steps against the same tokens one by one.

Projections are fp32 matrix products whose sums may be ordered differently for
one token than for several (relative 2^-20 at their widths); after that a
value on a border may round to the next bf16 number, half a step of 2^-8.  The
probabilities are compared in total variation: 2^-5 allows a few such steps in
each of the four layers."""
import importlib.util
import os

import pytest
import torch

from linear_attention_recurrence_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(cuda_device):
    build.build()
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_speculative_steps_equal_token_by_token(example):
    N, K, steps = 5, 3, 6
    fast = example.HybridStack(N, max_tokens=64, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(7)
    first = torch.arange(N, device="cuda", dtype=torch.int32)
    last, history = first, [[int(t)] for t in first]
    for _ in range(steps):
        counts, tokens, last = fast.step(last, K, gen)
        for n in range(N):
            history[n] += tokens[n, :int(counts[n])].tolist()
        assert ((counts >= 1) & (counts <= K + 1)).all()
    assert fast.lens.tolist() == [len(h) - 1 for h in history]
    assert binding.kda_last_device_status() == 0
    # every request by itself, one token at a time
    probs = fast.forward(last[:, None])[0][:, 0]
    for n in range(N):
        slow = example.HybridStack(N, max_tokens=64, seed=3)
        one = torch.ones(N, dtype=torch.int32, device="cuda")
        for t in history[n]:
            p, inputs = slow.forward(torch.full((N, 1), t, dtype=torch.int32, device="cuda"))
            if slow.lens[n] < len(history[n]) - 1:
                slow.commit(inputs, one)
        assert float((p[n, 0] - probs[n]).abs().sum()) / 2 < 2 ** -5
        for a, b in zip(fast.held, slow.held):
            if isinstance(a, torch.Tensor):
                assert float((a[n] - b[n]).norm() / b[n].norm()) < 2 ** -5


def test_the_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["hybrid_decode.py", "--requests", "3", "--steps", "4"])
    example.main()
    assert "device status 0" in capsys.readouterr().out
