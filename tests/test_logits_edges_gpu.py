"""kda_logits_probs in place, with rows apart, and with what has been said seen to count, where the tests beside this one
leave something out.  Bounds as in test_logits_gpu.py."""
import importlib.util
import os

import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from test_logits_gpu import TYPES, check, logits_of, reference, rules

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# rows that start with a vector or not, one tile of a CTA's or more, one row or many
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,R,V", [(1, 1, 1), (2, 3, 5), (3, 2, 2049), (2, 4, 50021), (1, 3, 131077), (1, 2, 300007), (1, 2, 409600),
                                   (40, 8, 9001)])
def test_in_place(N, R, V, dtype):
    x = logits_of(N, R, V, dtype, V).cuda()
    u = {n: t.cuda() for n, t in rules(N, R, V, 60, 9, True, V).items()}
    want = kda.kda_logits_probs(x, out_dtype=dtype, **u)
    for _ in range(3):
        held = x.clone()
        assert kda.kda_logits_probs(held, out=held, **u) is held
        assert torch.equal(held, want)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("V,stride,first", [(50021, 50048, 0), (5003, 5008, 0), (5003, 5005, 1), (4096, 4104, 0), (4096, 4099, 3),
                                            (131077, 131104, 0), (300007, 300032, 8)])
def test_rows_further_apart_than_they_are_long(V, stride, first, dtype, out_dtype):
    x = logits_of(2, 3, stride + first, dtype, V)
    x[..., :first] = x[..., first + V:] = float("nan")  # nothing of what lies between rows is seen
    check(x.cuda()[..., first:first + V], rules(2, 3, V, 50, 5, True, V), out_dtype)


def test_a_stack_penalises_all_that_has_been_said():
    """The example's stack: its history, the token that it runs over, and the drafts before a row."""
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    stack = example.HybridStack(1, "l", vocabulary=50, max_tokens=32, seed=5, repetition=4.0)
    tokens = torch.tensor([[7, 20, 31]], dtype=torch.int32, device="cuda")
    stack.lens.fill_(2)
    stack.said[0, :2] = torch.tensor([9, 11], device="cuda")
    seen = []

    def with_logits(logits, **kw):
        seen.append((logits, kw))
        return kda.kda_logits_probs(logits, **kw)

    example.kda_logits_probs = with_logits
    got, _ = stack.forward(tokens)
    (logits, _), = seen
    said = [[9, 11, 7], [9, 11, 7, 20], [9, 11, 7, 20, 31]]
    x = logits.double().cpu()
    for r, ids in enumerate(said):
        for t in ids:
            x[0, r, t] = x[0, r, t] / 4 if x[0, r, t] > 0 else x[0, r, t] * 4
    want = torch.softmax(x, -1)
    # an exponent is off by a few half-steps of its size (some units), and so is p: 2^-18 covers both with room
    assert ((got.double().cpu() - want).abs() <= 2.0 ** -18 * want).all()
    free, _ = reference(logits.cpu(), {})
    for r, ids in enumerate(said):  # the rule shows at each of them: beside the others, all have become less likely
        others = [t for t in range(50) if t not in ids]
        kept = float((got[0, r, others].double().cpu() / free[0, r, others]).mean())
        assert all(float(got[0, r, t]) < 0.999 * kept * float(free[0, r, t]) for t in ids)
