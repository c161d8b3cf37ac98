"""Acceptance of drafted tokens: whole numbers, equal to the definition
evaluated sequence by sequence in 64 bits."""
import math

import pytest
import torch

from linear_attention_recurrence_fwd_gb300 import binding, build

pytestmark = pytest.mark.gpu
F32, BF, FP = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    build.build()


def pick(w, u):
    w = torch.where((w > 0) & (w < math.inf), w, torch.zeros_like(w))
    total = torch.cumsum(w, 0)
    if not float(total[-1]) > 0:
        return -1
    at = torch.nonzero(total > u * total[-1])
    return int(at[0]) if at.numel() else int(torch.nonzero(w > 0)[-1])


def reference(toks, draft, target, uniform, lens):
    N, K1, V = target.shape
    u = uniform.double()
    counts, out = [], []
    for n in range(N):
        row = [-1] * K1
        m = K1 - 1 if lens is None else min(int(lens[n]), K1 - 1)
        if m < 0:
            counts.append(0)
            out.append(row)
            continue
        a = 0
        while a < m:
            t = int(toks[n, a])
            if not 0 <= t < V:
                break
            q = 1.0 if draft is None else float(draft[n, a, t])
            if not float(u[n, a]) * q < float(target[n, a, t]):
                break
            row[a] = t
            a += 1
        p = target[n, a].double()
        w = p
        if a < m:
            if draft is not None:
                w = p - draft[n, a].double()
            else:
                w = p.clone()
                if 0 <= int(toks[n, a]) < V:
                    w[int(toks[n, a])] = 0
        row[a] = pick(w, float(u[n, K1 - 1]))
        if row[a] < 0:
            row[a] = pick(p, float(u[n, K1 - 1]))
        counts.append(a + 1)
        out.append(row)
    return torch.tensor(counts, dtype=torch.int32), torch.tensor(out, dtype=torch.int32).view(N, K1)


def make(N, K, V, dtype=F32, seed=0, near=0.5):
    g = torch.Generator().manual_seed(seed)
    z = 3 * torch.randn((N, K + 1, V), generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :K] + near * torch.randn((N, K, V), generator=g), -1)
    toks = torch.multinomial(q.reshape(N * K, V), 1, generator=g).view(N, K).int() if K else torch.zeros((N, 0), dtype=torch.int32)
    return toks, q.to(dtype), p.to(dtype), torch.rand((N, K + 1), generator=g)


def check(toks, draft, target, uniform, lens=None, flagged=False):
    up = lambda t: None if t is None else t.cuda()
    binding.kda_last_device_status()
    counts, out = binding.kda_draft_accept(up(toks), up(draft), up(target), up(uniform), draft_lens=up(lens))
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == (1 if flagged else 0)
    rc, ro = reference(toks, draft, target, uniform, lens)
    assert torch.equal(counts.cpu(), rc)
    assert torch.equal(out.cpu(), ro)
    return rc, ro


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("N,K,V", [(1, 1, 1), (3, 2, 2), (5, 4, 31), (7, 3, 1000), (4, 5, 4096),
                                   (9, 7, 32771), (2, 4, 131072), (40, 1, 257)])
def test_sizes_and_types(N, K, V, dtype):
    check(*make(N, K, V, dtype, seed=N + V))


def test_many_sequences():
    rc, _ = check(*make(400, 3, 999, seed=2))
    assert rc.min() == 1 and rc.max() == 4


@pytest.mark.parametrize("near", [0.0, 5.0])
def test_all_kept_and_hardly_any(near):
    rc, _ = check(*make(30, 4, 5000, near=near, seed=9))
    assert (rc == 5).all() if near == 0 else (rc == 1).any()


def test_without_draft_probabilities():
    toks, _, p, u = make(50, 3, 700, seed=3)
    check(toks, None, p, u)
    hot = torch.zeros_like(p).scatter_(2, torch.nn.functional.pad(toks, (0, 1))[..., None].long(), 1.0)
    rc, _ = check(toks, None, hot, u)  # the target is certain of every draft
    assert (rc == 4).all()


def test_no_drafts_draws_from_the_target():
    toks, q, p, u = make(20, 0, 3001, seed=4)
    rc, _ = check(toks, None, p, u)
    assert (rc == 1).all()


def test_draft_lengths_and_idle_sequences():
    toks, q, p, u = make(9, 4, 333, seed=5)
    lens = torch.tensor([-1, 0, 1, 2, 3, 4, 9, -100, 2], dtype=torch.int32)
    check(toks, q, p, u, lens)
    check(toks, None, p, u, lens)


def test_extreme_random_numbers():
    toks, q, p, u = make(12, 3, 2049, seed=6)
    check(toks, q, p, torch.zeros_like(u))
    check(toks, q, p, torch.full_like(u, 1 - 2.0 ** -24))


def test_zero_probabilities_at_the_ends():
    """A running sum passes only at an entry that has weight."""
    toks, q, p, u = make(6, 1, 4000, seed=7)
    p[:, :, :1500] = 0
    p[:, :, 3000:] = 0
    check(toks, q, p, torch.zeros_like(u))
    check(toks, q, p, torch.full_like(u, 1 - 2.0 ** -24))


def test_no_positive_weight_falls_back_to_the_target():
    """The draft's probability is the larger everywhere; the draft itself has none."""
    toks, q, p, u = make(4, 1, 500, seed=8)
    toks.fill_(3)
    p[:, 0, 3] = 0
    q = p[:, :1] * 2
    rc, _ = check(toks, q, p, u)
    assert (rc == 1).all()


def test_no_probability_at_all():
    toks, q, p, u = make(3, 2, 100, seed=8)
    p.zero_()
    rc, ro = check(toks, q, p, u)
    assert (ro == -1).all() and (rc == 1).all()


def test_infinite_and_nan_probabilities_have_no_weight():
    toks, q, p, u = make(5, 2, 3000, seed=10)
    toks.clamp_(min=10)
    p[:, :, 4] = math.nan
    p[:, :, 5] = math.inf
    q[:, :, 6] = math.nan
    q[:, :, 7] = math.inf
    check(toks, q, p, u)


def test_drafts_outside_the_vocabulary_are_flagged():
    toks, q, p, u = make(4, 3, 200, seed=11)
    toks[1, 0], toks[2, 1] = 200, -1
    check(toks, q, p, torch.zeros_like(u), flagged=True)
    check(toks, None, p, torch.zeros_like(u), flagged=True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strided_and_oddly_aligned_rows(dtype):
    N, K, V = 5, 3, 1201
    toks, q, p, u = make(N, K, V, dtype, seed=12)
    wide_p = torch.zeros((N, K + 3, V + 6), dtype=dtype)
    wide_q = torch.zeros((N + 1, K + 1, V + 9), dtype=dtype)
    wide_p[:, 1:K + 2, 3:V + 3], wide_q[1:, :K, 5:V + 5] = p, q
    rc, ro = reference(toks, q, p, u, None)
    counts, out = binding.kda_draft_accept(toks.cuda(), wide_q.cuda()[1:, :K, 5:V + 5],
                                           wide_p.cuda()[:, 1:K + 2, 3:V + 3], u.cuda())
    assert torch.equal(counts.cpu(), rc) and torch.equal(out.cpu(), ro)


def test_offsets_beyond_32_bits():
    """Sequences 2^31 + 8 elements apart."""
    toks, q, p, u = make(2, 1, 3000, BF, seed=13)
    step = (1 << 31) + 8
    buf = torch.empty(step + 6000, dtype=BF, device="cuda")
    view = buf.as_strided((2, 2, 3000), (step, 3000, 1))
    view.copy_(p.cuda())
    counts, out = binding.kda_draft_accept(toks.cuda(), q.cuda(), view, u.cuda())
    rc, ro = reference(toks, q, p, u, None)
    assert torch.equal(counts.cpu(), rc) and torch.equal(out.cpu(), ro)


def test_distribution_is_the_targets():
    """The first token gained over 40000 sequences of one (p, q): the share of
    each of 8 tokens is within 5 standard deviations of the target's."""
    N, V = 40000, 8
    g = torch.Generator().manual_seed(14)
    p, q = torch.softmax(torch.randn((2, V), generator=g), -1)
    toks = torch.multinomial(q, N, replacement=True, generator=g).view(N, 1).int()
    u = torch.rand((N, 2), generator=g)
    _, out = binding.kda_draft_accept(toks.cuda(), q.expand(N, 1, V).contiguous().cuda(),
                                      p.expand(N, 2, V).contiguous().cuda(), u.cuda())
    share = torch.bincount(out[:, 0].cpu().long(), minlength=V) / N
    assert ((share - p).abs() <= 5 * torch.sqrt(p * (1 - p) / N)).all()


def test_other_stream_and_graph():
    toks, q, p, u = (x.cuda() for x in make(6, 3, 5000, seed=15))
    counts, out = binding.kda_draft_accept(toks, q, p, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c2, o2 = binding.kda_draft_accept(toks, q, p, u, stream=side)
    side.synchronize()
    assert torch.equal(counts, c2) and torch.equal(out, o2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c3, o3 = binding.kda_draft_accept(toks, q, p, u)
    for _ in range(2):
        c3.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(counts, c3) and torch.equal(out, o3)


def test_no_sequences():
    c, t = binding.kda_draft_accept(torch.empty((0, 2), dtype=torch.int32, device="cuda"), None,
                                    torch.empty((0, 3, 10), device="cuda"), torch.empty((0, 3), device="cuda"))
    assert c.shape == (0,) and t.shape == (0, 3)


@pytest.mark.parametrize("V", [2048, 2049, 3000, 4096, 6144, 8192])
@pytest.mark.parametrize("N", [1, 300])
def test_sequences_of_several_blocks_with_nothing_before_their_sums(N, V):
    """No drafts to look at and slices of few or no entries: the blocks of a
    sequence exchange their sums as soon as they have started."""
    toks, q, p, u = make(N, 0, V, seed=V + N)
    for lens in (None, (torch.arange(N) % 3 - 1).int()):  # idle sequences among them
        check(toks, None, p, u, lens)
    toks, q, p, u = make(N, 2, V, seed=V + N + 1)
    check(toks, q, p, u, (torch.arange(N) % 4 - 1).int())
