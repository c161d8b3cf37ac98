"""New tokens into a paged cache with the position rotation, against fp64."""
import math

import pytest
import torch

from linear_attention_recurrence_fwd_gb300 import binding, build
from cache_cases import HALF, assert_within

pytestmark = pytest.mark.gpu
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
MARK = 7.0  # in every row of the pool before the call


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    build.build()


def freqs(rot, base=10000.0):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def rotate(x, pos, inv_freq, interleaved):
    """[T, H, d] fp64 turned by pos * inv_freq, as products of complex numbers."""
    half = 0 if inv_freq is None else inv_freq.numel()
    if half == 0:
        return x.clone()
    y = x.clone()
    turn = torch.polar(torch.ones(1, half, dtype=torch.float64), pos.double()[:, None] * inv_freq)[:, None]
    if interleaved:
        z = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
        y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def tolerance(y, x, dtype, scale):
    """Half a step of the stored type, and the fp32 turn: the angle is held to
    2^-24 of a half turn, sine and cosine to 2^-23, two products and a sum."""
    v = (y / scale).abs()
    turn = 2.0 ** -20 * x.abs().amax(-1, keepdim=True) / scale
    least = 2.0 ** -10 if dtype == E4 else 2.0 ** -25 if dtype == FP else 0.0  # half the smallest subnormal
    return (v * HALF[dtype]).clamp(min=least) + 2 * turn


def check(lens, K, Hq=4, Hkv=2, d=128, page=16, act=BF, dtype=None, rot=None, interleaved=False,
          layout="token", counts=None, packed=None, fused=True, k_scale=1.0, v_scale=1.0, seed=0,
          mult=1.0, base=10000.0):
    dtype = act if dtype is None else dtype
    rot = d if rot is None else rot
    g = torch.Generator().manual_seed(seed)
    new = [K] * len(lens) if packed is None else packed
    T = sum(new)
    x = mult * torch.randn((T, (Hq + 2 * Hkv) * d), generator=g)
    x = x.to(act).cuda()
    if fused:
        q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([Hq * d, Hkv * d, Hkv * d], 1))
    else:
        q, k, v = (y.contiguous().unflatten(1, (-1, d)) for y in x.split([Hq * d, Hkv * d, Hkv * d], 1))
    first = [n // page for n in lens]
    last = [(n + m - 1) // page for n, m in zip(lens, new)]
    need = [max(0, b - a + 1) for a, b in zip(first, last)]
    total = sum(need) + 2
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max([0] + last) + 1), -1, dtype=torch.int32)
    at = 0
    for n, m in enumerate(need):
        table[n, first[n]:first[n] + m] = order[at:at + m]
        at += m
    shape = (total, Hkv, page, d) if layout == "head" else (total, page, Hkv, d)
    kp, vp = (torch.full(shape, MARK).to(dtype).cuda() for _ in range(2))
    if layout == "head":
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    cache = binding.PagedCache(kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                               k_scale=k_scale, v_scale=v_scale)
    inv = freqs(rot, base) if rot else None
    lead = (len(lens), K)
    kw = dict(q=q, inv_freq=None if inv is None else inv.cuda(), interleaved=interleaved)
    if packed is None:
        kw["q"] = q.unflatten(0, lead)
        if counts is not None:
            kw["counts"] = torch.tensor(counts, dtype=torch.int32).cuda()
        qo = binding.kda_cache_append(k.unflatten(0, lead), v.unflatten(0, lead), cache, **kw).flatten(0, 1)
    else:
        edges = [0]
        for m in packed:
            edges.append(edges[-1] + m)
        qo = binding.kda_cache_append(k, v, cache, cu_seqlens=torch.tensor(edges, dtype=torch.int32).cuda(), **kw)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 0
    # the expected pools, fp64, and which rows were written
    pos = torch.cat([torch.arange(m) + n for n, m in zip(lens, new)]) if T else torch.zeros(0, dtype=torch.long)
    seq = torch.cat([torch.full((m,), n) for n, m in enumerate(new)]) if T else pos
    num = torch.cat([torch.arange(m) for m in new]) if T else pos
    xq, xk, xv = (y.double().cpu() for y in (q, k, v))
    rq, rk = rotate(xq, pos, inv, interleaved), rotate(xk, pos, inv, interleaved)
    assert_within(qo, rq, tolerance(rq, xq, act, 1.0), "q")
    keep = torch.ones(T, dtype=torch.bool) if counts is None else num < torch.tensor(counts)[seq]
    page_of, row = table[seq, pos // page].long()[keep], (pos % page)[keep]
    for got, y, src, scale, name in ((kp, rk, xk, k_scale, "k"), (vp, xv, xv, v_scale, "v")):
        got = got.float().cpu()
        lim = 448.0 if dtype == E4 else math.inf
        assert_within(got[page_of, row], (y[keep] / scale).clamp(-lim, lim),
                      tolerance(y[keep], src[keep], dtype, scale), name)
        got[page_of, row] = MARK
        assert (got == MARK).all(), f"{name}: rows of other tokens were written"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("act,dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types(act, dtype, d, interleaved):
    check([0, 1, 15, 16, 300], 3, d=d, act=act, dtype=dtype, interleaved=interleaved,
          k_scale=0.5 if dtype == E4 else 1.0, v_scale=0.3 if dtype == E4 else 1.0)


@pytest.mark.parametrize("rot", [0, 2, 16, 30, 64, 126])
@pytest.mark.parametrize("interleaved", [False, True])
def test_partial_rotation(rot, interleaved):
    check([0, 7, 100], 2, rot=rot, interleaved=interleaved, seed=rot)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (32, 8), (5, 1), (16, 16)])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_head_layouts(Hq, Hkv, layout):
    check([3, 50], 4, Hq=Hq, Hkv=Hkv, layout=layout, d=64, fused=Hq != 5)


@pytest.mark.parametrize("page", [1, 3, 16, 48, 1000])
def test_page_sizes(page):
    check([0, 47, 48, 200], 9, page=page, d=64, seed=page)


def test_far_positions():
    """Angles of many turns: base 2 keeps every frequency high."""
    check([999_983, 1 << 20, (1 << 24) + 1], 5, page=64, base=2.0)
    check([999_983, 123_457], 5, page=64)


def test_counts():
    check([5, 30, 100, 0], 4, counts=[0, 4, 2, 1])


@pytest.mark.parametrize("packed", [[1], [5, 0, 1, 40], [0, 0, 3], [130, 1, 77]])
def test_packed_prompts(packed):
    check([17 * n for n in range(len(packed))], 0, packed=packed)


def test_many_sequences():
    check([(31 * n) % 700 for n in range(300)], 1, Hq=2, Hkv=1, d=64)


def test_eight_bit_saturation_and_small_values():
    check([0, 40], 8, dtype=E4, rot=0, mult=300.0, k_scale=0.5, v_scale=1.0)
    check([0, 40], 8, dtype=E4, rot=0, mult=0.01)


def test_queries_in_place_and_without_queries():
    d, K = 128, 2
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn((1, K, 2, d), generator=g).to(BF).cuda() for _ in range(2))
    pools = [torch.zeros((2, 16, 2, d), dtype=BF, device="cuda") for _ in range(2)]
    cache = binding.PagedCache(*pools, torch.tensor([[1]], dtype=torch.int32).cuda(),
                               torch.tensor([3], dtype=torch.int32).cuda())
    inv = freqs(d).cuda()
    want = binding.kda_cache_append(k, k, cache, q=q, inv_freq=inv)
    first = cache.k_pages.clone()
    assert binding.kda_cache_append(k, k, cache, inv_freq=inv) is None
    assert torch.equal(first, cache.k_pages)
    got = binding.kda_cache_append(k, k, cache, q=q, inv_freq=inv, q_out=q)
    assert got is q and torch.equal(got, want)


def test_pages_and_positions_outside_are_left_out_and_flagged():
    d = 64
    k = torch.ones((4, 1, 1, d), dtype=BF, device="cuda")
    pools = [torch.full((2, 16, 1, d), MARK, dtype=BF, device="cuda") for _ in range(2)]
    table = torch.tensor([[0], [2], [-1], [1]], dtype=torch.int32).cuda()
    binding.kda_last_device_status()
    cache = binding.PagedCache(*pools, table, torch.tensor([4, 4, 4, 16], dtype=torch.int32).cuda())
    binding.kda_cache_append(k, k, cache)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 1
    assert (cache.k_pages[0, 4] == 1).all()
    cache.k_pages[0, 4] = MARK
    assert (cache.k_pages == MARK).all()
    cache.lens.copy_(torch.tensor([-1, -1, -1, -1], dtype=torch.int32))
    binding.kda_cache_append(k, k, cache)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 1
    assert (cache.k_pages == MARK).all()


@pytest.mark.parametrize("edges", [[0, 2, 4], [1, 3, 6], [0, 9, 6], [-3, 2, 6], [4, 1, 6]])
def test_offsets_that_are_none_are_flagged(edges):
    """T = 6 rows; rows without a sequence, or all, are left out; nothing is written elsewhere."""
    d = 64
    k = torch.ones((6, 1, d), dtype=BF, device="cuda")
    pools = [torch.full((3, 16, 1, d), MARK, dtype=BF, device="cuda") for _ in range(2)]
    table = torch.tensor([[0], [1]], dtype=torch.int32).cuda()
    binding.kda_last_device_status()
    cache = binding.PagedCache(*pools, table, torch.tensor([0, 0], dtype=torch.int32).cuda())
    binding.kda_cache_append(k, k, cache, cu_seqlens=torch.tensor(edges, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 1
    assert (cache.k_pages[2] == MARK).all()


def test_other_stream_and_graph():
    d, K = 128, 2
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn((2, K, 2, d), generator=g).to(BF).cuda() for _ in range(2))
    pools = [torch.zeros((4, 16, 2, d), dtype=BF, device="cuda") for _ in range(2)]
    cache = binding.PagedCache(*pools, torch.tensor([[1, 0], [2, 3]], dtype=torch.int32).cuda(),
                               torch.tensor([15, 3], dtype=torch.int32).cuda())
    inv = freqs(d).cuda()
    want = binding.kda_cache_append(k, k, cache, q=q, inv_freq=inv)
    pages = cache.k_pages.clone()
    cache.k_pages.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.kda_cache_append(k, k, cache, q=q, inv_freq=inv, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(cache.k_pages, pages)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = binding.kda_cache_append(k, k, cache, q=q, inv_freq=inv)
        cache.lens.add_(1)
    cache.k_pages.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(cache.k_pages, pages)
    assert cache.lens.tolist() == [16, 4]


def test_no_tokens():
    pools = [torch.zeros((1, 16, 1, 64), dtype=BF, device="cuda") for _ in range(2)]
    cache = binding.PagedCache(*pools, torch.zeros((1, 1), dtype=torch.int32).cuda(),
                               torch.zeros(1, dtype=torch.int32).cuda())
    k = torch.empty((1, 0, 1, 64), dtype=BF, device="cuda")
    assert binding.kda_cache_append(k, k, cache, q=k).shape == k.shape
