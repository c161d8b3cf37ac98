"""Calls of several host threads at once, each on a stream of its own."""
import ctypes
import threading

import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from linear_attention_recurrence_fwd_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [(409600, 140000), (409593, 131105), (40000, 60000, 100000)])
def test_probabilities_of_different_vocabularies(sizes):
    """They need different amounts of shared memory for the counts of one kernel.  Straight to the library, two threads
    for each size, so that calls meet often."""
    lib, start, jobs, codes = binding.load(), threading.Barrier(2 * len(sizes)), [], []
    for V in sizes * 2:
        x = torch.randn((1, 1, V), generator=torch.Generator().manual_seed(V)).cuda()
        u = {"tokens": torch.arange(50, dtype=torch.int32, device="cuda")[None], "repetition": torch.full((1,), 1.3, device="cuda")}
        want, got, stream = kda.kda_logits_probs(x, **u), torch.empty_like(x), torch.cuda.Stream()
        rules = binding._LogitsRules(tokens=u["tokens"].data_ptr(), repetition=u["repetition"].data_ptr(), tokens_stride=50, L=50)
        args = (x.data_ptr(), binding.KDA_F32, V, V, ctypes.addressof(rules), got.data_ptr(), binding.KDA_F32, 1, 1, V, stream.cuda_stream)
        jobs.append((args, want, got, stream, x, u, rules))
    torch.cuda.synchronize()

    def work(args):
        start.wait()
        codes.extend({lib.kda_logits_probs(*args) for _ in range(8000)})

    threads = [threading.Thread(target=work, args=(job[0],)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert set(codes) == {0}
    for _, want, got, *_ in jobs:
        assert torch.equal(want, got)
