"""kda_logits_probs against its rules in 64 bits, row by row.

Bounds.  An entry x is off by a few half-steps of fp32 of what it was added up from (|x| and the penalties and
biases given), and p by that over the temperature, plus the exponent's own rounding (2^-24 of its size, twice)
and 2^-21 for the exponential, the sum and the quotient; then half a step of the output's type.  The
exponential flushes what is below 2^-126 of the row's largest."""
import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from linear_attention_recurrence_fwd_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
         (torch.float16, torch.float32), (torch.float16, torch.float16)]


def bits(mask, V):
    """bool [.., V] to int32 words."""
    words = (V + 31) // 32
    m = torch.nn.functional.pad(mask, (0, 32 * words - V)).unflatten(-1, (words, 32)).long()
    w = (m << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def rules(N, R, V, L=0, J=0, mask=False, seed=0, penalties=True, temperature=True):
    g = torch.Generator().manual_seed(seed)
    u = {}
    if R > 1:
        u["drafts"] = torch.randint(-1, V + 1, (N, R - 1), generator=g, dtype=torch.int32)
    if L:
        # few different tokens, so that many come often; some outside the vocabulary
        u["tokens"] = torch.randint(-2, min(V, 50) + 2, (N, L), generator=g, dtype=torch.int32)
        u["tokens"][:, ::7] = V - 1
        u["lens"] = torch.randint(-1, L + 3, (N,), generator=g, dtype=torch.int32)
        u["prompt_lens"] = torch.randint(-1, L + 2, (N,), generator=g, dtype=torch.int32)
    if penalties:
        u["repetition"] = 0.8 + 0.6 * torch.rand(N, generator=g)
        u["presence"] = torch.randn(N, generator=g)
        u["frequency"] = 0.2 * torch.randn(N, generator=g)
    if J:
        u["bias_ids"] = torch.randint(-1, V + 1, (N, J), generator=g, dtype=torch.int32)
        u["bias_ids"][:, J // 2:] = u["bias_ids"][:, :J - J // 2].clone()  # each twice
        u["bias"] = torch.randn((N, J), generator=g)
    if mask:
        u["mask"] = bits(torch.rand((N, R, V), generator=g) < 0.5, V)
    if temperature:
        u["temperature"] = 0.3 + torch.rand(N, generator=g)
    return u


def reference(logits, u):
    """(probabilities, how far each entry of x may be off in half-steps of fp32)."""
    N, R, V = logits.shape
    out, size = torch.zeros((N, R, V), dtype=torch.float64), torch.zeros((N, R, V), dtype=torch.float64)
    for n in range(N):
        one = lambda name, default: float(u[name][n]) if u.get(name) is not None else default  # noqa: B023,E731
        tokens = u["tokens"][n].tolist() if u.get("tokens") is not None else []
        L = max(0, min(len(tokens), int(u["lens"][n]) if u.get("lens") is not None else len(tokens)))
        P = int(u["prompt_lens"][n]) if u.get("prompt_lens") is not None else 0
        said, new = torch.zeros(V, dtype=torch.bool), torch.zeros(V, dtype=torch.float64)
        for i, t in enumerate(tokens[:L]):
            if 0 <= t < V:
                said[t] = True
                new[t] += i >= P
        extra, weight = torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.float64)
        if u.get("bias") is not None:
            for t, b in zip(u["bias_ids"][n].tolist(), u["bias"][n].tolist()):
                if 0 <= t < V:
                    extra[t] += b
                    weight[t] += abs(b)
        for r in range(R):
            if r and u.get("drafts") is not None and 0 <= int(u["drafts"][n, r - 1]) < V:
                said[int(u["drafts"][n, r - 1])] = True
                new[int(u["drafts"][n, r - 1])] += 1
            x = logits[n, r].double()
            rep, fall = one("repetition", 1.0), one("frequency", 0.0) * new + one("presence", 0.0) * (new > 0)
            x = torch.where(said, torch.where(x > 0, x / rep, x * rep), x)
            size[n, r] = 8 * (x.abs() + abs(one("frequency", 0.0)) * new + abs(one("presence", 0.0)) + weight)
            x = x - fall + extra
            if u.get("mask") is not None:
                m = u["mask"].expand(N, R, -1)[n, r].long()
                t = torch.arange(V)
                x = torch.where((m[t // 32] >> (t % 32)) & 1 == 1, x, -torch.inf)
            T = one("temperature", 1.0)
            if not (x > -torch.inf).any() and not torch.isnan(x).any():
                continue
            if T > 0:
                out[n, r] = torch.softmax(x / T, -1)
                size[n, r] = (size[n, r] + 3 * (x - x.max()).abs()) / T
            else:
                out[n, r, int(x.argmax())] = 1
    return out, size


def check(logits, u, out_dtype=torch.float32, **kw):
    dev = {k: v.cuda() for k, v in u.items()}
    got = kda.kda_logits_probs(logits.cuda() if not logits.is_cuda else logits, out_dtype=out_dtype, **dev, **kw)
    assert got.dtype == out_dtype and got.shape == logits.shape
    ref, size = reference(logits.cpu(), u)
    e = torch.finfo(out_dtype).eps / 2
    tiny = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}[out_dtype]
    size = torch.nan_to_num(size, 0, 0, 0)
    top = (size * 2.0 ** -24 * ref).sum(-1, keepdim=True)  # what the sum is off by
    bound = ref * (e + 2.0 ** -21 + 2 * (size * 2.0 ** -24) + 2 * top) + 2 * tiny
    assert ((got.double().cpu() - ref).abs() <= bound).all(), float(((got.double().cpu() - ref).abs() / bound).max())
    return got


def logits_of(N, R, V, dtype, seed=0):
    return (4 * torch.randn((N, R, V), generator=torch.Generator().manual_seed(seed))).to(dtype)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("N,R,V,L,J,mask", [(1, 1, 1, 0, 0, False), (1, 1, 7, 3, 1, True), (2, 3, 1000, 40, 5, True),
                                            (3, 2, 4099, 200, 31, True), (1, 4, 16384, 700, 33, False),
                                            (2, 1, 20000, 10, 100, True), (1, 2, 50021, 1000, 7, True)])
def test_rules(N, R, V, L, J, mask, dtype, out_dtype):
    check(logits_of(N, R, V, dtype, V), rules(N, R, V, L, J, mask, V), out_dtype)


@pytest.mark.parametrize("V", [101, 4099, 20001])
def test_biases_of_an_earlier_call_stay_there(V):
    # Rows that start between vectors: the first vector holds entries before the row.  The earlier call leaves a full
    # list of biases, of entries that the later one has and gives none for, in every SM's shared memory.
    before = {"bias_ids": torch.arange(992, dtype=torch.int32).remainder(96).repeat(600, 1), "bias": torch.full((600, 992), 3.0)}
    x = logits_of(600, 1, 128, torch.float32, 3)
    u = {"bias_ids": torch.tensor([[50]], dtype=torch.int32), "bias": torch.tensor([[0.5]])}
    for dtype in (torch.float32, torch.bfloat16):
        kda.kda_logits_probs(x.cuda(), **{k: v.cuda() for k, v in before.items()})
        check(logits_of(1, 8, V, dtype, V), u)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [131072, 131080, 200000, 262145, 300000, 409600])
def test_large_vocabularies(V, dtype):
    check(logits_of(1, 2, V, dtype, V), rules(1, 2, V, 300, 9, True, V), torch.float32)


def test_many_rows():
    check(logits_of(90, 5, 6000, torch.float32, 1), rules(90, 5, 6000, 60, 4, True, 1))
    check(logits_of(40, 9, 33000, torch.bfloat16, 2), rules(40, 9, 33000, 20, 2, False, 2), torch.bfloat16)


def test_beyond_the_counted_vocabulary():
    V = 600001
    u = rules(1, 1, V, 0, 3, True, 4, penalties=False)
    check(logits_of(1, 1, V, torch.float32, 4), u)
    with pytest.raises(binding.KDAError) as e:
        kda.kda_logits_probs(logits_of(1, 1, V, torch.float32).cuda(), repetition=torch.ones(1, device="cuda"))
    assert e.value.code == 2


@pytest.mark.parametrize("name", ["tokens", "lens", "prompt_lens", "repetition", "presence", "frequency", "drafts", "mask",
                                  "temperature", "bias"])
def test_each_rule_left_out(name):
    u = rules(3, 3, 2000, 50, 6, True, 5)
    for n in {"tokens": ("tokens", "lens", "prompt_lens"), "bias": ("bias", "bias_ids")}.get(name, (name,)):
        del u[n]
    check(logits_of(3, 3, 2000, torch.float32, 5), u)


def test_more_biases_than_the_list_holds():
    check(logits_of(2, 2, 3000, torch.float32, 6), rules(2, 2, 3000, 0, 2500, False, 6, penalties=False))


@pytest.mark.parametrize("V", [1000, 40001])
def test_temperature_zero(V):
    x = logits_of(6, 2, V, torch.float32, 7)
    x[0, 0, 17] = x[0, 0, V - 2] = 50.0  # a tie: the first
    x[1, 1, V - 1] = 60.0
    x[3, 0, 5] = float("nan")
    u = rules(6, 2, V, 20, 3, False, 7)
    u["temperature"] = torch.tensor([0.0, 0.0, -1.0, 0.0, 0.5, float("nan")])
    u = {n: t for n, t in u.items() if n not in ("bias", "bias_ids", "tokens", "lens", "prompt_lens", "drafts")}
    got = kda.kda_logits_probs(x.cuda(), **{n: t.cuda() for n, t in u.items()}).cpu()
    for n in (0, 1, 2, 5):
        for r in range(2):
            want = torch.zeros(V)
            want[int(x[n, r].argmax())] = 1
            assert torch.equal(got[n, r], want), (n, r)
    assert got[0, 0, 17] == 1
    assert torch.isnan(got[3, 0]).all() and not torch.isnan(got[3, 1]).any()


@pytest.mark.parametrize("V", [1000, 40001])
def test_masked_rows_and_values_that_are_not_finite(V):
    x = logits_of(1, 8, V, torch.float32, 8)
    allowed = torch.ones((1, 8, V), dtype=torch.bool)
    allowed[0, 0] = False                                    # nothing is left
    x[0, 1] = -torch.inf                                     # nothing either
    x[0, 2, 3:] = -torch.inf                                 # three entries
    x[0, 3, 10], allowed[0, 3, 10] = float("nan"), False     # behind a mask
    x[0, 4, 10], allowed[0, 4, 10] = float("inf"), False
    x[0, 5, 10] = float("nan")                               # in sight
    x[0, 6, 10] = float("inf")
    x[0, 7] = torch.finfo(torch.float32).min                 # all equal
    got = kda.kda_logits_probs(x.cuda(), mask=bits(allowed, V).cuda()).cpu()
    assert (got[0, :2] == 0).all()
    assert torch.allclose(got[0, 2, :3].double(), torch.softmax(x[0, 2, :3].double(), -1), rtol=1e-6) and (got[0, 2, 3:] == 0).all()
    for r in (3, 4):
        want = torch.softmax(x[0, r].double().masked_fill(~allowed[0, r], -torch.inf), -1)
        assert torch.allclose(got[0, r].double(), want, rtol=1e-5) and got[0, r, 10] == 0
    assert torch.isnan(got[0, 5]).all() and torch.isnan(got[0, 6]).all()
    assert torch.allclose(got[0, 7], torch.full((V,), 1 / V), rtol=1e-6)


def test_small_temperatures_and_large_logits():
    x = logits_of(4, 1, 5000, torch.float32, 9)
    x[1] *= 1e6
    u = {"temperature": torch.tensor([1e-3, 0.7, 1e-30, 1e30])}
    got = kda.kda_logits_probs(x.cuda(), temperature=u["temperature"].cuda()).cpu()
    assert torch.isfinite(got).all()
    assert torch.allclose(got.double().sum(-1), torch.ones(4, 1, dtype=torch.float64), atol=1e-5)
    assert got[2, 0, int(x[2, 0].argmax())] == 1
    assert torch.allclose(got[3, 0], torch.full((5000,), 1 / 5000), rtol=1e-5)


def test_shared_masks_strides_and_in_place():
    N, R, V = 3, 2, 2048
    x = logits_of(N, R + 1, V + 64, torch.float32, 10).cuda()
    u = rules(N, R, V, 30, 3, False, 10)
    for shape in ((1, 1), (N, 1), (1, R), (N, R)):
        u["mask"] = bits(torch.rand((*shape, V)) < 0.5, V)
        view = x[:, 1:, :V]
        got = check(view, u)
        wide = torch.zeros((*u["mask"].shape[:2], 100), dtype=torch.int32)
        wide[..., :V // 32] = u["mask"]
        same = kda.kda_logits_probs(view, **{n: (wide.cuda()[..., :V // 32] if n == "mask" else t.cuda()) for n, t in u.items()})
        assert torch.equal(got, same)
    u["tokens"] = torch.nn.functional.pad(u["tokens"], (0, 5))
    dev = {n: t.cuda() for n, t in u.items()}
    dev["tokens"] = dev["tokens"][:, :30]
    held = x[:, 1:, :V].contiguous()
    want = kda.kda_logits_probs(held, **dev)
    assert kda.kda_logits_probs(held, out=held, **dev) is held
    assert torch.equal(held, want)
    odd = x[:, 1:, 1:V]  # rows that start at odd addresses
    u = rules(N, R, V - 1, 30, 3, True, 11)
    check(odd, u)


def test_repeats_streams_and_graphs():
    N, R, V = 4, 3, 33000
    x = logits_of(N, R, V, torch.float32, 12).cuda()
    u = {n: t.cuda() for n, t in rules(N, R, V, 500, 5, True, 12).items()}
    want = kda.kda_logits_probs(x, **u)
    assert torch.equal(want, kda.kda_logits_probs(x, **u))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = kda.kda_logits_probs(x, stream=stream, **u)
    stream.synchronize()
    assert torch.equal(want, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = kda.kda_logits_probs(x, **u)
    x.copy_(logits_of(N, R, V, torch.float32, 13).cuda())
    u["lens"].fill_(17)
    graph.replay()
    assert torch.equal(held, kda.kda_logits_probs(x, **u))


def test_into_draft_acceptance():
    """Logits to tokens: a request's drafts are judged by the probabilities after penalties and masks."""
    N, K, V = 5, 3, 1500
    x = logits_of(N, K + 1, V, torch.float32, 14)
    u = rules(N, K + 1, V, 40, 3, True, 14)
    u["drafts"] = u["drafts"].clamp(0, V - 1)
    dev = {n: t.cuda() for n, t in u.items()}
    probs = kda.kda_logits_probs(x.cuda(), **dev)
    uniform = torch.rand((N, K + 1)).cuda()
    counts, tokens = kda.kda_draft_accept(dev["drafts"], None, probs, uniform)
    p, (ref, _) = probs.cpu(), reference(x, u)
    for n in range(N):
        a = 0
        while a < K and float(uniform[n, a]) < float(p[n, a, u["drafts"][n, a]]):
            a += 1
        assert int(counts[n]) == a + 1
        assert ref[n, a, int(tokens[n, a])] > 0  # never a masked one


def test_arguments_are_checked():
    x = torch.zeros((2, 3, 100), device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for kw in (dict(tokens=i32(3, 4)), dict(tokens=torch.zeros((2, 4), device="cuda")), dict(lens=i32(2)),
               dict(drafts=i32(2, 3)), dict(repetition=torch.ones(3, device="cuda")), dict(bias=torch.ones((2, 3), device="cuda")),
               dict(bias_ids=i32(2, 3), bias=torch.ones((2, 4), device="cuda")), dict(mask=i32(2, 3, 3)), dict(mask=i32(2, 2, 4)),
               dict(temperature=torch.ones(2)), dict(out_dtype=torch.bfloat16), dict(out=torch.zeros((2, 3, 99), device="cuda"))):
        with pytest.raises(ValueError):
            kda.kda_logits_probs(x, **kw)
    for bad in (x.double(), x[0], x.transpose(1, 2), x.cpu()):
        with pytest.raises(ValueError):
            kda.kda_logits_probs(bad)
    assert kda.kda_logits_probs(x[:0]).shape == (0, 3, 100)
