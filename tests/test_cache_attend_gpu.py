"""Attention of the newest tokens over a paged cache, against fp64.

Every position that a token must not see holds NaN (unowned rows and pages),
so a masked value that reached an output would show."""
import math

import pytest
import torch

from linear_attention_recurrence_fwd_gb300 import binding, build
from cache_cases import NAN, assert_within, attend_reference, make_cache

pytestmark = pytest.mark.gpu
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_device):
    build.build()


def check(lens, K=1, Hq=4, Hkv=2, d=128, page=16, act=BF, dtype=None, window=0, counts=None,
          layout="token", scale=None, k_scale=1.0, v_scale=1.0, seed=0, mult=1.5, **kw):
    dtype = act if dtype is None else dtype
    cache, keys, values = make_cache(lens, K, Hkv, d, page, dtype, seed, layout, k_scale=k_scale,
                                     v_scale=v_scale)
    g = torch.Generator().manual_seed(seed + 1)
    q = (mult * torch.randn((len(lens), K, Hq, d), generator=g)).to(act)
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    out, lse = binding.kda_cache_attend(q.cuda(), cache, scale=scale, window=window, counts=cnt,
                                        return_lse=True, **kw)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 0
    ref, rlse, tol, ltol = attend_reference(q, keys, values, lens, counts,
                                            d ** -0.5 if scale is None else scale, window)
    assert_within(lse, rlse, ltol, "lse")
    assert_within(out, ref, tol, "out")
    return cache, q, out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("act,dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
def test_types_and_head_dims(act, dtype, d):
    check([0, 1, 2, 15, 16, 63, 64, 65, 200], act=act, dtype=dtype, d=d,
          k_scale=0.5 if dtype == E4 else 1.0, v_scale=0.25 if dtype == E4 else 1.0)


@pytest.mark.parametrize("Hq,Hkv,K", [(1, 1, 1), (5, 5, 1), (7, 1, 1), (8, 2, 1), (16, 1, 1), (17, 1, 1),
                                      (32, 2, 1), (12, 3, 3), (8, 1, 5), (32, 2, 4), (33, 1, 2),
                                      (16, 2, 9), (14, 2, 5), (64, 1, 3)])
def test_head_layouts_and_rows(Hq, Hkv, K):
    check([0, 3, 70, 129, 300], K=K, Hq=Hq, Hkv=Hkv, seed=Hq + K)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 48, 64, 100, 128, 1000])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_page_sizes_and_layouts(page, layout):
    check([0, 62, 63, 64, 99, 100, 511], K=2, page=page, layout=layout, d=64, seed=page)


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 5000])
@pytest.mark.parametrize("K", [1, 4])
def test_windows(window, K):
    check([0, 1, 16, 63, 64, 130, 700], K=K, window=window, seed=window)


@pytest.mark.parametrize("K,counts", [(1, [0, 1, 0, 1]), (5, [0, 5, 2, 1]), (3, [3, 0, 0, 0])])
def test_rows_that_see_nothing(K, counts):
    cache, q, out, lse = check([0, 100, 64, 300], K=K, counts=counts)
    for n, c in enumerate(counts):
        assert (out[n, c:] == 0).all() and (lse[n, c:] == -math.inf).all()


def test_negative_lengths_see_nothing_or_little():
    # position lens + i: -1, 0, 1 for the first sequence, none for the others
    check([-1, -3, -100], K=3)


def test_one_long_sequence():
    check([70001], Hq=8, Hkv=1, page=64)


def test_long_and_short_sequences_together():
    check([20000, 0, 5, 9000, 1, 1, 33, 12345], K=2, Hq=8, Hkv=2, page=32, seed=5)


def test_many_sequences():
    lens = [(37 * n) % 1500 for n in range(300)]
    check(lens, Hq=2, Hkv=1, d=64, page=16)


def test_max_len_is_a_bound_and_may_be_short():
    _, _, out, _ = check([100, 2000, 7], Hq=4, Hkv=1, max_len=2001)
    _, _, other, _ = check([100, 2000, 7], Hq=4, Hkv=1, max_len=10)
    assert torch.allclose(out.float(), other.float(), atol=2 ** -6)


def test_large_scores_and_equal_scores():
    check([500], Hq=4, Hkv=1, mult=30.0, scale=1.0)   # one position takes nearly all
    check([500], Hq=4, Hkv=1, mult=0.0)               # every position the same


def test_projection_slice_as_queries():
    lens, K, Hq, d = [5, 80], 3, 4, 128
    cache, keys, values = make_cache(lens, K, 2, d, 16, BF)
    fused = torch.randn((2 * K, (Hq + 4) * d), generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    q = fused[:, :Hq * d].unflatten(1, (Hq, d)).unflatten(0, (2, K))
    assert not q.is_contiguous()
    out = binding.kda_cache_attend(q, cache)
    ref, _, tol, _ = attend_reference(q, keys, values, lens, None, d ** -0.5, 0)
    assert_within(out, ref, tol, "out")


def test_infinite_and_nan_in_a_later_draft_do_not_reach_earlier_tokens():
    """Token 1 of 3 holds infinities and NaN: token 0 must not notice, tokens 1 and 2 must."""
    lens, K, d = [70], 3, 128
    cache, keys, values = make_cache(lens, K, 1, d, 16, BF)
    pos = lens[0] + 1
    page = int(cache.block_table[0, pos // 16])
    q = torch.randn((1, K, 2, d), generator=torch.Generator().manual_seed(4)).to(BF)
    for bad in (NAN, math.inf):
        cache.v_pages[page, pos % 16] = bad
        cache.k_pages[page, pos % 16] = 0
        out = binding.kda_cache_attend(q.cuda(), cache)
        ref, _, tol, _ = attend_reference(q[:, :1], [keys[0][:lens[0] + 1]], [values[0][:lens[0] + 1]],
                                          lens, None, d ** -0.5, 0)
        assert_within(out[:, :1], ref, tol, "token 0")
        assert not torch.isfinite(out[:, 1:].float()).any()


def test_nan_before_the_window_stays_out():
    lens, d = [300], 64
    cache, keys, values = make_cache(lens, 1, 1, d, 16, BF)
    for x in (cache.k_pages, cache.v_pages):
        for p in range(0, 251):  # positions 251.. are seen (window 50)
            x[int(cache.block_table[0, p // 16]), p % 16] = NAN
    q = torch.randn((1, 1, 2, d), generator=torch.Generator().manual_seed(4)).to(BF)
    out = binding.kda_cache_attend(q.cuda(), cache, window=50)
    ref, _, tol, _ = attend_reference(q, keys, values, lens, None, d ** -0.5, 50)
    assert_within(out, ref, tol, "out")


def test_offsets_beyond_32_bits():
    """Three pages 2^31 - 128 elements apart (an 8-bit cache of 6 GB)."""
    Hkv, d, page, step = 1, 128, 16, (1 << 31) - 128
    bufs = [torch.empty(2 * step + page * Hkv * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pools = [b.view(E4).as_strided((3, page, Hkv, d), (step, Hkv * d, d, 1)) for b in bufs]
    g = torch.Generator().manual_seed(6)
    toks = [torch.randn((48, Hkv, d), generator=g).to(E4) for _ in range(2)]
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    for pool, tok in zip(pools, toks):
        for j, p in enumerate(table[0].tolist()):
            pool[p].copy_(tok[16 * j:16 * j + 16].cuda())
    cache = binding.PagedCache(*pools, table.cuda(), torch.tensor([46], dtype=torch.int32).cuda())
    q = torch.randn((1, 1, 4, d), generator=g).to(BF)
    out = binding.kda_cache_attend(q.cuda(), cache)
    ref, _, tol, _ = attend_reference(q, [toks[0].double()], [toks[1].double()], [46], None, d ** -0.5, 0)
    assert_within(out, ref, tol, "out")


def test_pages_outside_the_pool_are_left_out_and_flagged():
    lens, d = [100, 40], 128
    cache, keys, values = make_cache(lens, 1, 1, d, 16, BF)
    binding.kda_last_device_status()
    cache.block_table[0, 2] = 10 ** 6
    cache.block_table[0, 4] = -7
    q = torch.randn((2, 1, 2, d), generator=torch.Generator().manual_seed(4)).to(BF)
    out = binding.kda_cache_attend(q.cuda(), cache)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 1
    kept = [j for j in range(101) if j // 16 not in (2, 4)]
    ref, _, tol, _ = attend_reference(q, [keys[0][kept], keys[1]], [values[0][kept], values[1]],
                                      [len(kept) - 1, 40], None, d ** -0.5, 0)
    assert_within(out, ref, tol, "out")


def test_lengths_beyond_the_table_are_clamped_and_flagged():
    lens, d = [31, 5], 64
    cache, keys, values = make_cache(lens, 1, 1, d, 16, BF)
    cache.lens[0] = 1000  # the table holds 32 positions
    q = torch.randn((2, 1, 2, d), generator=torch.Generator().manual_seed(4)).to(BF)
    out = binding.kda_cache_attend(q.cuda(), cache)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 1
    ref, _, tol, _ = attend_reference(q, keys, values, lens, None, d ** -0.5, 0)
    assert_within(out, ref, tol, "out")


def test_other_stream_repeats_and_graph():
    """The same bits on another stream, on a second call, and from a graph
    whose lens change between replays."""
    lens, K = [3000, 17, 600], 2
    cache, keys, values = make_cache(lens, K, 2, 128, 16, BF)
    q = torch.randn((3, K, 8, 128), generator=torch.Generator().manual_seed(8)).to(BF).cuda()
    first = binding.kda_cache_attend(q, cache)
    assert torch.equal(first, binding.kda_cache_attend(q, cache))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = binding.kda_cache_attend(q, cache, stream=side)
    side.synchronize()
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.kda_cache_attend(q, cache)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    cache.lens.copy_(torch.tensor([1999, 16, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ref, _, tol, _ = attend_reference(q.cpu(), keys, values, [1999, 16, 0], None, 128 ** -0.5, 0)
    assert_within(out, ref, tol, "replayed")


def test_no_sequences_and_no_tokens():
    cache, _, _ = make_cache([], 1, 2, 64, 16, BF)
    assert binding.kda_cache_attend(torch.empty((0, 1, 2, 64), dtype=BF, device="cuda"), cache).shape == (0, 1, 2, 64)
    cache, _, _ = make_cache([5], 0, 2, 64, 16, BF)
    assert binding.kda_cache_attend(torch.empty((1, 0, 2, 64), dtype=BF, device="cuda"), cache).shape == (1, 0, 2, 64)


# More query rows to a key head than one row tile: 20, 32, 33, 40, 48, 49 and 100 of them.
MANY = [(1, 20, 1), (4, 16, 2), (3, 11, 1), (5, 32, 4), (3, 16, 1), (7, 7, 1), (25, 4, 1)]


@pytest.mark.parametrize("K,Hq,Hkv", MANY)
@pytest.mark.parametrize("act,dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows(K, Hq, Hkv, act, dtype, d):
    check([0, 1, 63, 127, 128, 129, 700], K=K, Hq=Hq, Hkv=Hkv, d=d, act=act, dtype=dtype, page=32, seed=K,
          k_scale=0.5 if dtype == E4 else 1.0, v_scale=0.25 if dtype == E4 else 1.0)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("window", [1, 5, 64, 129, 1000])
def test_many_rows_windows_counts_and_layouts(window, dtype):
    check([0, 30, 200, 511, 1000, 3], K=5, Hq=16, Hkv=2, window=window, counts=[5, 0, 3, 5, 1, 2], page=48,
          layout="head", dtype=dtype, seed=window)


@pytest.mark.parametrize("dtype", [BF, E4])
def test_many_rows_long_and_negative(dtype):
    check([20000, -2, 5, 9000, 0, 33], K=4, Hq=10, Hkv=1, page=64, dtype=dtype, seed=3)
    check([40000], K=5, Hq=32, Hkv=4, page=64, dtype=dtype, seed=4)


@pytest.mark.parametrize("dtype", [BF, E4])
def test_many_rows_scores_that_keep_growing(dtype):
    """Keys that grow along the sequence: the running maximum is passed again and again."""
    lens, K, Hq, d = [1000], 3, 12, 128
    cache, keys, values = make_cache(lens, K, 1, d, 64, dtype)
    grow = torch.linspace(0.05, 8.0, lens[0] + K)[:, None, None]
    new = (keys[0].float() * grow).to(dtype).float()
    for p in range(lens[0] + K):
        cache.k_pages[int(cache.block_table[0, p // 64]), p % 64] = new[p].to(dtype).cuda()
    q = (2 * torch.randn((1, K, Hq, d), generator=torch.Generator().manual_seed(2))).to(BF)
    out, lse = binding.kda_cache_attend(q.cuda(), cache, return_lse=True)
    ref, rlse, tol, ltol = attend_reference(q, [new.double()], values, lens, None, d ** -0.5, 0)
    assert_within(lse, rlse, ltol, "lse")
    assert_within(out, ref, tol, "out")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [70, 127, 128])
@pytest.mark.parametrize("dtype", [BF, FP, E4])
def test_many_rows_infinite_and_nan_in_a_later_draft(dtype, at, d):
    """As above with 40 rows; positions before, at and after a tile's border."""
    lens, K, Hq = [at - 1], 5, 8
    act = FP if dtype == FP else BF
    cache, keys, values = make_cache(lens, K, 1, d, 16, dtype)
    pos = lens[0] + 1
    page = int(cache.block_table[0, pos // 16])
    q = torch.randn((1, K, Hq, d), generator=torch.Generator().manual_seed(4)).to(act)
    for bad in (NAN, math.inf) if dtype != E4 else (NAN,):
        cache.v_pages[page, pos % 16] = torch.full((1, d), bad).to(dtype).cuda()
        cache.k_pages[page, pos % 16] = torch.zeros((1, d)).to(dtype).cuda()
        out = binding.kda_cache_attend(q.cuda(), cache)
        ref, _, tol, _ = attend_reference(q[:, :1], [keys[0][:lens[0] + 1]], [values[0][:lens[0] + 1]],
                                          lens, None, d ** -0.5, 0)
        assert_within(out[:, :1], ref, tol, "token 0")
        assert not torch.isfinite(out[:, 1:].float()).any()


def test_one_infinite_value_of_a_later_draft_reaches_its_channel_alone():
    lens, K, Hq, d = [100], 4, 8, 128
    cache, keys, values = make_cache(lens, K, 1, d, 16, BF)
    pos = lens[0] + 2
    cache.v_pages[int(cache.block_table[0, pos // 16]), pos % 16, 0, 77] = math.inf
    values[0][pos, 0, 77] = 0  # the other channels' reference
    q = torch.randn((1, K, Hq, d), generator=torch.Generator().manual_seed(4)).to(BF)
    out = binding.kda_cache_attend(q.cuda(), cache)
    ref, _, tol, _ = attend_reference(q, keys, values, lens, None, d ** -0.5, 0)
    rest = [c for c in range(d) if c != 77]
    assert_within(out[..., rest], ref[..., rest], tol[..., rest], "other channels")
    assert (out[:, 2:, :, 77] == math.inf).all()
    assert torch.isfinite(out[:, :2].float()).all()


@pytest.mark.parametrize("rows", [4, 40])
@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_at_every_row_count(rows, dtype, d):
    lens = [300]
    cache, keys, values = make_cache(lens, 1, 1, d, 16, dtype)
    binding.kda_last_device_status()
    for j, bad in ((0, -1), (7, 10 ** 9), (15, cache.k_pages.shape[0])):
        cache.block_table[0, j] = bad
    q = torch.randn((1, 1, rows, d), generator=torch.Generator().manual_seed(4)).to(BF)
    out = binding.kda_cache_attend(q.cuda(), cache)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 1
    kept = [j for j in range(301) if j // 16 not in (0, 7, 15)]
    ref, _, tol, _ = attend_reference(q, [keys[0][kept]], [values[0][kept]], [len(kept) - 1], None, d ** -0.5, 0)
    assert_within(out, ref, tol, "out")


@pytest.mark.parametrize("page", [1, 3, 5])
@pytest.mark.parametrize("Hq", [4, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_odd_pages_of_an_8_bit_cache(page, Hq, d):
    check([0, 62, 300], Hq=Hq, Hkv=1, d=d, page=page, dtype=E4, seed=page)


@pytest.mark.parametrize("Hq", [4, 40])
def test_strides_of_interleaved_keys_and_values(Hq):
    """Keys and values as the two halves of one pool, pages [page, 2, token, head, d]."""
    lens, d = [130, 7], 128
    cache, keys, values = make_cache(lens, 1, 1, d, 16, BF)
    pool = torch.stack([cache.k_pages, cache.v_pages], 1).contiguous()
    both = binding.PagedCache(pool[:, 0], pool[:, 1], cache.block_table, cache.lens)
    q = torch.randn((2, 1, Hq, d), generator=torch.Generator().manual_seed(4)).to(BF)
    out = binding.kda_cache_attend(q.cuda(), both)
    ref, _, tol, _ = attend_reference(q, keys, values, lens, None, d ** -0.5, 0)
    assert_within(out, ref, tol, "out")


def test_many_rows_repeat_and_follow_the_lengths_in_a_graph():
    lens, K = [3000, 17, 600], 3
    cache, keys, values = make_cache(lens, K, 2, 128, 16, BF)
    q = torch.randn((3, K, 16, 128), generator=torch.Generator().manual_seed(8)).to(BF).cuda()
    first = binding.kda_cache_attend(q, cache)
    for _ in range(3):
        assert torch.equal(first, binding.kda_cache_attend(q, cache))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.kda_cache_attend(q, cache)
    cache.lens.copy_(torch.tensor([1999, 16, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ref, _, tol, _ = attend_reference(q.cpu(), keys, values, [1999, 16, 0], None, 128 ** -0.5, 0)
    assert_within(out, ref, tol, "replayed")


@pytest.mark.parametrize("Hq", [4, 40])
def test_pages_whose_rows_are_interleaved(Hq):
    """Rows of all pages side by side ([row, page, head, d]), and one page with odd strides of its own."""
    lens, d = [130, 7], 128
    cache, keys, values = make_cache(lens, 1, 2, d, 16, BF)
    q = torch.randn((2, 1, Hq, d), generator=torch.Generator().manual_seed(4)).to(BF)
    pools = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (cache.k_pages, cache.v_pages)]
    assert pools[0].stride(0) < pools[0].stride(1)
    out = binding.kda_cache_attend(q.cuda(), binding.PagedCache(*pools, cache.block_table, cache.lens))
    ref, _, tol, _ = attend_reference(q, keys, values, lens, None, d ** -0.5, 0)
    assert_within(out, ref, tol, "out")
    # one page, one head: the strides of those dimensions say nothing
    cache, keys, values = make_cache([9], 1, 1, d, 16, BF, spare=0)
    pools = [x.as_strided((1, 16, 1, d), (3, d, 5, 1)) for x in (cache.k_pages, cache.v_pages)]
    odd = binding.PagedCache(*pools, cache.block_table, cache.lens)
    out = binding.kda_cache_attend(q[:1].cuda(), odd)
    ref, _, tol, _ = attend_reference(q[:1], keys, values, [9], None, d ** -0.5, 0)
    assert_within(out, ref, tol, "out")


@pytest.mark.parametrize("length", [40, 5000])
@pytest.mark.parametrize("rows", [4, 40])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_nan_in_a_query_reaches_its_own_row_alone(dtype, rows, length):
    """A row all of whose scores are NaN has no maximum; it must not pass for one that sees nothing."""
    K, Hq, d = (1, 4, 128) if rows == 4 else (5, 8, 128)
    cache, keys, values = make_cache([length], K, 1, d, 64, dtype)
    q = torch.randn((1, K, Hq, d), generator=torch.Generator().manual_seed(4)).to(BF)
    q[0, 0, 1, 3] = NAN
    out, lse = binding.kda_cache_attend(q.cuda(), cache, return_lse=True)
    assert torch.isnan(out[0, 0, 1].float()).all() and torch.isnan(lse[0, 0, 1])
    q[0, 0, 1] = 0
    ref, rlse, tol, ltol = attend_reference(q, keys, values, [length], None, d ** -0.5, 0)
    out[0, 0, 1], lse[0, 0, 1] = ref[0, 0, 1], rlse[0, 0, 1]
    assert_within(lse, rlse, ltol, "lse")
    assert_within(out, ref, tol + 2.0 ** -8 * ref.abs(), "out")


@pytest.mark.parametrize("act", [BF, FP])
def test_many_rows_8_bit_queries_of_all_sizes(act):
    """Rows whose entries lie far apart, and rows far above and below the others."""
    K, Hq, d, lens = 5, 8, 128, [700]
    cache, keys, values = make_cache(lens, K, 1, d, 64, E4)
    g = torch.Generator().manual_seed(9)
    q = torch.randn((1, K, Hq, d), generator=g) * 2.0 ** torch.randint(-12, 1, (1, K, Hq, d), generator=g)
    q = (q * 2.0 ** torch.randint(-10, 4, (1, K, Hq, 1), generator=g)).to(act)
    out, lse = binding.kda_cache_attend(q.cuda(), cache, return_lse=True)
    ref, rlse, tol, ltol = attend_reference(q, keys, values, lens, None, d ** -0.5, 0)
    assert_within(lse, rlse, ltol, "lse")
    assert_within(out, ref, tol, "out")


def test_many_rows_8_bit_many_small_weights_beside_a_large_one():
    """One score 2^20 times the weight of each of 60000 others: together they still count."""
    K, Hq, d, length = 5, 8, 128, 60000
    cache, keys, values = make_cache([length], K, 1, d, 64, E4)
    k = torch.zeros_like(cache.k_pages, dtype=torch.float32)
    page = int(cache.block_table[0, 0])
    k[page, 5, 0, 0] = 16.0
    cache.k_pages.copy_(k.to(E4))
    keys[0].zero_()
    keys[0][5, 0, 0] = 16.0
    q = torch.zeros((1, K, Hq, d))
    q[..., 0] = 13.875 / 16 * d ** 0.5
    q = q.to(BF)
    out, lse = binding.kda_cache_attend(q.cuda(), cache, return_lse=True)
    ref, rlse, tol, ltol = attend_reference(q, keys, values, [length], None, d ** -0.5, 0)
    assert_within(lse, rlse, ltol, "lse")
    assert_within(out, ref, tol, "out")


# A large bound on the lengths keeps short sequences on the units of up to 48 rows.
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("act,dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("K,Hq", [(5, 8), (4, 8), (13, 4), (8, 8)])
def test_many_rows_short_sequences_with_a_large_bound(K, Hq, act, dtype, d):
    check([0, 1, 70, 127, 128, 200], K=K, Hq=Hq, Hkv=1, d=d, act=act, dtype=dtype, max_len=9000)
    check([5, 300], K=K, Hq=Hq, Hkv=1, d=d, act=act, dtype=dtype, max_len=9000, window=33, counts=[K, 2], page=3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [70, 127, 128])
@pytest.mark.parametrize("dtype", [BF, FP, E4])
def test_many_rows_nan_in_a_later_draft_with_a_large_bound(dtype, at, d):
    lens, K, Hq = [at - 1], 5, 8
    cache, keys, values = make_cache(lens, K, 1, d, 16, dtype)
    pos = lens[0] + 1
    page = int(cache.block_table[0, pos // 16])
    q = torch.randn((1, K, Hq, d), generator=torch.Generator().manual_seed(4)).to(FP if dtype == FP else BF)
    for bad in (NAN, math.inf) if dtype != E4 else (NAN,):
        cache.v_pages[page, pos % 16] = torch.full((1, d), bad).to(dtype).cuda()
        cache.k_pages[page, pos % 16] = torch.zeros((1, d)).to(dtype).cuda()
        out = binding.kda_cache_attend(q.cuda(), cache, max_len=9000)
        ref, _, tol, _ = attend_reference(q[:, :1], [keys[0][:lens[0] + 1]], [values[0][:lens[0] + 1]],
                                          lens, None, d ** -0.5, 0)
        assert_within(out[:, :1], ref, tol, "token 0")
        assert not torch.isfinite(out[:, 1:].float()).any()


@pytest.mark.parametrize("dtype", [BF, E4])
def test_nan_in_a_query_with_a_large_bound(dtype):
    cache, _, _ = make_cache([40], 5, 1, 128, 64, dtype)
    q = torch.randn((1, 5, 8, 128), generator=torch.Generator().manual_seed(4)).to(BF)
    q[0, 0, 1, 3] = NAN
    out, lse = binding.kda_cache_attend(q.cuda(), cache, return_lse=True, max_len=9000)
    assert torch.isnan(out[0, 0, 1].float()).all() and torch.isnan(lse[0, 0, 1])
    lse[0, 0, 1] = 0
    assert torch.isfinite(lse).all() and torch.isfinite(out[:, 1:].float()).all()


@pytest.mark.parametrize("rows", [4, 40])
@pytest.mark.parametrize("act,dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
def test_small_weights_beside_a_large_one_without_a_value(act, dtype, rows):
    """The first position takes nearly all the weight and holds zeros; the others, 2^-26 of it each,
    are the whole output.  Enough units for every block to hold whole sequences."""
    N, Hkv, d, length = 40, 8, 128, 999
    cache, keys, values = make_cache([length] * N, 1, Hkv, d, 16, dtype)
    for x in (cache.k_pages, cache.v_pages):
        x.copy_(torch.zeros(x.shape).to(dtype))
    g = torch.Generator().manual_seed(3)
    for n in range(N):
        v = (64 * torch.randn((length + 1, Hkv, d), generator=g).abs()).to(dtype)
        v[0] = 0
        held = cache.block_table[n].long()
        at = torch.arange(length + 1, device="cuda")
        flat = cache.v_pages.view(torch.uint8) if dtype == E4 else cache.v_pages
        flat[held[at // 16], at % 16] = (v.view(torch.uint8) if dtype == E4 else v).cuda()
        cache.k_pages[int(held[0]), 0, :, 0] = 16.0
        keys[n].zero_()
        keys[n][0, :, 0] = 16.0
        values[n] = v.double()
    q = torch.zeros((N, 1, Hkv * rows, d))
    q[..., 0] = 1.0
    scale = 26 * math.log(2) / 16  # the first score is 26 in powers of two, the others 0
    out, lse = binding.kda_cache_attend(q.to(act).cuda(), cache, scale=scale, return_lse=True)
    ref, rlse, tol, ltol = attend_reference(q.to(act), keys, values, [length] * N, None, scale, 0)
    assert_within(lse, rlse, ltol, "lse")
    assert_within(out, ref, tol, "out")


@pytest.mark.parametrize("lens,window,max_len", [([40], 0, 0), ([40], 0, 9000), ([5000], 0, 0), ([625, 1137], 500, 0),
                                                 ([625, 1137], 500, 9000)])
@pytest.mark.parametrize("rows", [4, 13])
@pytest.mark.parametrize("act,dtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
def test_scores_of_minus_infinity_are_not_positions_that_are_not_seen(act, dtype, rows, lens, window, max_len):
    """A row all of whose scores overflow to -infinity is 0 / 0, with a sum of 0; the rows beside it see
    equal scores.  (With the window, the first tile is seen by the first two tokens alone.)"""
    K, d = 3, 128
    cache, keys, values = make_cache(lens, K, 1, d, 16, dtype)
    for n in range(len(lens)):
        at = torch.arange(lens[n] + K, device="cuda")
        k = torch.zeros((lens[n] + K, 1, d))
        k[..., 0] = -8
        flat = cache.k_pages.view(torch.uint8) if dtype == E4 else cache.k_pages
        flat[cache.block_table[n].long()[at // 16], at % 16] = (k.to(dtype).view(torch.uint8) if dtype == E4 else k.to(dtype)).cuda()
        keys[n] = k.double()
    q = torch.zeros((len(lens), K, rows, d))
    q[:, :, 1, 0] = 8.0
    out, lse = binding.kda_cache_attend(q.to(act).cuda(), cache, scale=1e38, window=window, max_len=max_len, return_lse=True)
    assert torch.isnan(out[:, :, 1].float()).all()
    assert (lse[:, :, 1] == -math.inf).all()
    q[:, :, 1] = 0
    ref, rlse, tol, ltol = attend_reference(q.to(act), keys, values, lens, None, 1e38, window)
    rest = [r for r in range(rows) if r != 1]
    assert_within(lse[:, :, rest], rlse[:, :, rest], ltol[:, :, rest], "lse")
    assert_within(out[:, :, rest], ref[:, :, rest], tol[:, :, rest], "out")


@pytest.mark.parametrize("length", [40, 5000])
@pytest.mark.parametrize("rows", [4, 40])
def test_an_infinite_query_over_an_8_bit_cache_gives_nan(rows, length):
    """Also where it would make every score -infinity."""
    d = 128
    cache, _, _ = make_cache([length], 1, 1, d, 16, E4)
    cache.k_pages.copy_(torch.full(cache.k_pages.shape, -1.0).to(E4))
    q = torch.zeros((1, 1, rows, d))
    q[0, 0, 2, 5] = math.inf
    out = binding.kda_cache_attend(q.to(BF).cuda(), cache, max_len=9000)
    assert torch.isnan(out[0, 0, 2].float()).all()
    rest = [r for r in range(rows) if r != 2]
    assert torch.isfinite(out[0, 0, rest].float()).all()


@pytest.mark.parametrize("rows", [4, 40])
def test_the_largest_bound_on_the_lengths_is_one(rows):
    """2^31 - 1, as for 'no bound': the launch and the workspace are those of any long sequence."""
    size = binding.load().kda_cache_attend_workspace_size
    most = (1 << 31) - 1
    assert size(3, 1, rows, 1, 128, most) == size(3, 1, rows, 1, 128, 1 << 30) == size(3, 1, rows, 1, 128, 1 << 20) > 0
    check([100, 2000, 7], Hq=rows, Hkv=1, max_len=most)


# Bad pages, strides and single infinities where the large bound puts 40 rows on the units of up to 48.
@pytest.mark.parametrize("bad", [(0, 7, 15), tuple(range(8, 16)), tuple(range(19))])
@pytest.mark.parametrize("act,dtype", [(BF, BF), (FP, FP), (BF, E4)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_bad_pages_with_a_large_bound(act, dtype, d, bad):
    """Single pages, a whole tile of 128 positions, and every page but the last one's drafts."""
    lens, K, Hq = [300], 5, 8
    cache, keys, values = make_cache(lens, K, 1, d, 16, dtype)
    binding.kda_last_device_status()
    for x, j in enumerate(bad):
        cache.block_table[0, j] = (-1, 10 ** 9, cache.k_pages.shape[0])[x % 3]
    q = torch.randn((1, K, Hq, d), generator=torch.Generator().manual_seed(4)).to(act)
    out, lse = binding.kda_cache_attend(q.cuda(), cache, max_len=9000, return_lse=True)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 1
    kept = [j for j in range(lens[0] + K) if j // 16 not in bad]
    ref, rlse, tol, ltol = attend_reference(q, [keys[0][kept]], [values[0][kept]], [len(kept) - K], None, d ** -0.5, 0)
    assert_within(lse, rlse, ltol, "lse")
    assert_within(out, ref, tol, "out")


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_bad_page_and_nan_in_a_later_draft_with_a_large_bound(dtype, d):
    """Both in one tile: the product formed row by row leaves the bad page out."""
    lens, K, Hq = [300], 5, 8
    cache, keys, values = make_cache(lens, K, 1, d, 16, dtype)
    binding.kda_last_device_status()
    cache.block_table[0, 17] = -1  # positions 272 to 287, in the tile of the drafts
    pos = lens[0] + 1
    page = int(cache.block_table[0, pos // 16])
    cache.v_pages[page, pos % 16] = torch.full((1, d), NAN).to(dtype).cuda()
    cache.k_pages[page, pos % 16] = torch.zeros((1, d)).to(dtype).cuda()
    q = torch.randn((1, K, Hq, d), generator=torch.Generator().manual_seed(4)).to(BF)
    out = binding.kda_cache_attend(q.cuda(), cache, max_len=9000)
    torch.cuda.synchronize()
    assert binding.kda_last_device_status() == 1
    kept = [j for j in range(lens[0] + 1) if j // 16 != 17]
    ref, _, tol, _ = attend_reference(q[:, :1], [keys[0][kept]], [values[0][kept]], [len(kept) - 1], None, d ** -0.5, 0)
    assert_within(out[:, :1], ref, tol, "token 0")
    assert not torch.isfinite(out[:, 1:].float()).any()


def test_many_rows_pages_that_no_entry_names_with_a_large_bound():
    """Every page bad: nothing is seen, in every row."""
    cache, _, _ = make_cache([200], 1, 1, 128, 16, BF)
    binding.kda_last_device_status()
    cache.block_table.fill_(-1)
    for rows in (4, 40):
        q = torch.randn((1, 1, rows, 128), generator=torch.Generator().manual_seed(4)).to(BF).cuda()
        out, lse = binding.kda_cache_attend(q, cache, max_len=9000, return_lse=True)
        torch.cuda.synchronize()
        assert binding.kda_last_device_status() == 1
        assert (out == 0).all() and (lse == -math.inf).all()


def test_many_rows_strides_with_a_large_bound():
    lens, d, Hq = [130, 7], 128, 80
    cache, keys, values = make_cache(lens, 1, 2, d, 16, BF)
    q = torch.randn((2, 1, Hq, d), generator=torch.Generator().manual_seed(4)).to(BF)
    ref, _, tol, _ = attend_reference(q, keys, values, lens, None, d ** -0.5, 0)
    pool = torch.stack([cache.k_pages, cache.v_pages], 1).contiguous()  # keys and values of a page side by side
    rows = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (cache.k_pages, cache.v_pages)]  # [row, page, head, d]
    for pools in ((pool[:, 0], pool[:, 1]), rows):
        out = binding.kda_cache_attend(q.cuda(), binding.PagedCache(*pools, cache.block_table, cache.lens), max_len=9000)
        assert_within(out, ref, tol, "out")


def test_many_rows_one_infinite_value_of_a_later_draft_with_a_large_bound():
    lens, K, Hq, d = [100], 5, 8, 128
    cache, keys, values = make_cache(lens, K, 1, d, 16, BF)
    pos = lens[0] + 2
    cache.v_pages[int(cache.block_table[0, pos // 16]), pos % 16, 0, 77] = math.inf
    values[0][pos, 0, 77] = 0  # the other channels' reference
    q = torch.randn((1, K, Hq, d), generator=torch.Generator().manual_seed(4)).to(BF)
    out = binding.kda_cache_attend(q.cuda(), cache, max_len=9000)
    ref, _, tol, _ = attend_reference(q, keys, values, lens, None, d ** -0.5, 0)
    rest = [c for c in range(d) if c != 77]
    assert_within(out[..., rest], ref[..., rest], tol[..., rest], "other channels")
    assert (out[:, 2:, :, 77] == math.inf).all()
    assert torch.isfinite(out[:, :2].float()).all()
