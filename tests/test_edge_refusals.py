"""Refusals at the edges of the calls' ranges, before anything is launched (no GPU; the pointers are never followed)."""
import ctypes

import pytest

from linear_attention_recurrence_fwd_gb300 import binding, build

F = ctypes.c_void_p(16)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_commits_take_aligned_counts(lib, off):
    at = ctypes.c_void_p(16 + off)
    assert lib.kda_linear_commit(F, F, 256, 256, F, 0, 2, 1, F, at, 3, 4, 2, 128, 128, None) == 3
    assert lib.kda_decode_commit(F, F, F, F, F, F, at, 3, 4, 2, 128, 128, None) == 3


@pytest.mark.parametrize("rules", [dict(tokens=16, repetition=16, L=(1 << 30) + 1), dict(tokens=16, repetition=16, L=(1 << 31) - 1),
                                   dict(bias_ids=16, bias=16, J=(1 << 30) + 1), dict(bias_ids=16, bias=16, J=(1 << 31) - 1)])
def test_histories_and_bias_lists_that_32_bits_do_not_count(lib, rules):
    u = binding._LogitsRules(**rules)
    assert lib.kda_logits_probs(F, 1, 100, 100, ctypes.addressof(u), F, 1, 1, 1, 100, None) == 2
