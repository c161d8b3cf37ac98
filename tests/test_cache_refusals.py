"""What the calls around a paged cache refuse, before any CUDA call: no GPU
is needed, and the fake pointers are never dereferenced."""
import ctypes

import pytest
import torch

from linear_attention_recurrence_fwd_gb300 import binding, build

F = 4096           # aligned fake pointer
BF16, F32, F16, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def cache(**kw):
    f = dict(k=F, v=F, block_table=F, lens=F, page_stride=16 * 2 * 128, token_stride=256, head_stride=128,
             table_stride=4, k_scale=1.0, v_scale=1.0, dtype=BF16, n_seq=3, num_pages=8, page_size=16,
             table_width=4, H_kv=2, d=128)
    f.update(kw)
    return binding._CacheStruct(**f)


BAD_CACHES = [(dict(n_seq=-1), 1), (dict(num_pages=-1), 1), (dict(page_size=0), 1), (dict(table_width=-1), 1),
              (dict(H_kv=0), 1), (dict(d=0), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(lens=None), 1),
              (dict(block_table=None), 1), (dict(k_scale=0.0), 1), (dict(v_scale=float("nan")), 1),
              (dict(page_stride=-8), 1), (dict(table_stride=-1), 1), (dict(dtype=F32), 2), (dict(dtype=F16), 2),
              (dict(dtype=9), 2), (dict(d=96), 2), (dict(d=256), 2), (dict(table_width=1 << 28), 2),
              (dict(k=F + 8), 3), (dict(v=F + 2), 3), (dict(page_stride=4), 3), (dict(token_stride=132), 3),
              (dict(head_stride=4), 3), (dict(dtype=E4M3, token_stride=264), 3)]


def append(lib, c=None, k=F, v=F, q=F, q_out=F, dtype=BF16, ks=512, vs=512, qs=512, qos=512, inv=F, rot=128,
           cu=None, counts=None, K=2, T=6, Hq=4):
    ref = None if c is False else ctypes.addressof(c or cache())
    return lib.kda_cache_append(ref, k, v, q, q_out, dtype, ks, vs, qs, qos, inv, rot, 0, cu, counts, K, T, Hq, None)


def attend(lib, c=None, q=F, dtype=BF16, qs=512, out=F, lse=F, counts=None, K=2, Hq=4, window=0, max_len=0,
           ws=None, wsb=0):
    ref = None if c is False else ctypes.addressof(c or cache())
    return lib.kda_cache_attend(ref, q, dtype, qs, out, lse, counts, K, Hq, 1.0, window, max_len, ws, wsb, None)


@pytest.mark.parametrize("fields,code", BAD_CACHES, ids=[str(sorted(f)[0]) + str(i) for i, (f, _) in enumerate(BAD_CACHES)])
def test_bad_caches(lib, fields, code):
    bad = cache(**fields)
    assert append(lib, bad) == code
    assert attend(lib, bad) == code


def test_append_arguments(lib):
    assert append(lib, False) == 1
    assert append(lib, k=None) == 1 and append(lib, v=None) == 1
    assert append(lib, q=None) == 1 and append(lib, q_out=None) == 1 and append(lib, Hq=0) == 1
    assert append(lib, T=5) == 1 and append(lib, T=-1) == 1 and append(lib, K=-2) == 1
    assert append(lib, cu=F, counts=F) == 1
    assert append(lib, rot=3) == 1 and append(lib, rot=130) == 1 and append(lib, inv=None) == 1
    assert append(lib, ks=-512) == 1
    assert append(lib, dtype=F32) == 2 and append(lib, dtype=E4M3) == 2
    assert append(lib, k=F + 8) == 3 and append(lib, q_out=F + 4) == 3 and append(lib, vs=516) == 3
    assert append(lib, inv=F + 4) == 3
    assert append(lib, K=0, T=0) == 0  # nothing to do


def test_append_rotated_queries_that_overlap(lib):
    assert append(lib, qos=0) == 1 and append(lib, qos=504) == 1
    assert append(lib, qos=0, K=0, T=0) == 0  # no two tokens


def test_attend_arguments(lib):
    assert attend(lib, False) == 1
    assert attend(lib, q=None) == 1 and attend(lib, out=None) == 1
    assert attend(lib, Hq=3) == 1 and attend(lib, Hq=0) == 1
    assert attend(lib, K=-1) == 1 and attend(lib, window=-1) == 1 and attend(lib, max_len=-1) == 1
    assert attend(lib, dtype=F32) == 2
    assert attend(lib, q=F + 8) == 3 and attend(lib, out=F + 8) == 3 and attend(lib, lse=F + 2) == 3
    assert attend(lib, qs=516) == 3
    assert attend(lib, K=0) == 0 and attend(lib, cache(n_seq=0)) == 0


def test_attend_workspace_size_of_nonsense_is_zero(lib):
    size = lib.kda_cache_attend_workspace_size
    assert size(0, 1, 4, 2, 128, 100) == 0 and size(1, 1, 3, 2, 128, 100) == 0
    assert size(1, 1, 4, 2, 96, 100) == 0 and size(1, 1, 4, 2, 128, -1) == 0


def test_attend_row_counts_past_32_bits(lib):
    big = (1 << 31) - 1
    assert attend(lib, cache(n_seq=1 << 22), K=1 << 22, Hq=1 << 20) == 2  # 2^64 rows
    assert attend(lib, cache(n_seq=big), K=big, Hq=big - 1) == 2
    assert attend(lib, cache(n_seq=1 << 15), K=1 << 10, Hq=64) == 2
    assert lib.kda_cache_attend_workspace_size(big, big, big, 1, 128, 100) == 0
    assert lib.kda_cache_attend_workspace_size(1, 1 << 20, 1 << 20, 1, 128, 100) == 0


def test_accept_arguments(lib):
    def call(toks=F, draft=F, target=F, dtype=F32, strides=(400, 100, 500, 100), u=F, lens=None, counts=F,
             out=F, N=2, K=4, V=100):
        return lib.kda_draft_accept(toks, draft, target, dtype, *strides, u, lens, counts, out, N, K, V, None)
    assert call(toks=None) == 1 and call(target=None) == 1 and call(u=None) == 1
    assert call(counts=None) == 1 and call(out=None) == 1
    assert call(N=-1) == 1 and call(K=-1) == 1 and call(V=0) == 1
    assert call(strides=(-1, 0, 0, 0)) == 1
    assert call(dtype=E4M3) == 2 and call(dtype=7) == 2
    assert call(target=F + 2) == 3 and call(draft=F + 1, dtype=BF16) == 3 and call(u=F + 1) == 3
    assert call(N=0) == 0


def test_host_tensors_are_refused():
    pages = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.PagedCache(pages, pages, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.kda_draft_accept(torch.zeros((1, 1), dtype=torch.int32), None, torch.zeros((1, 2, 4)), torch.zeros((1, 2)))


class Claimed:
    """A host tensor that says it is on a GPU: for what is looked at before any launch."""
    is_cuda = True

    def __init__(self, t, index=0):
        self._t, self._index = t, index
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self._index

    def __getattr__(self, name):
        return getattr(self._t, name)


def claimed_cache(N=3, width=4):
    pages = [Claimed(torch.zeros((5, 16, 2, 64), dtype=torch.bfloat16)) for _ in range(2)]
    return binding.PagedCache(*pages, Claimed(torch.zeros((N, width), dtype=torch.int32)),
                              Claimed(torch.zeros(N, dtype=torch.int32)))


def test_assignments_to_a_cache_are_followed():
    """What a call gets is the struct behind cache._ref."""
    c = claimed_cache()
    seen = binding._CacheStruct.from_address(c._ref)
    lens = Claimed(torch.ones(3, dtype=torch.int32))
    c.lens = lens
    assert c.lens is lens and seen.lens == lens.data_ptr()
    table = Claimed(torch.zeros((3, 9), dtype=torch.int32))
    c.block_table = table  # a grown table
    assert seen.block_table == table.data_ptr() and seen.table_width == 9 and seen.table_stride == 9
    assert c.capacity == 9 * 16
    c.k_scale, c.v_scale = 0.5, 0.25
    assert (seen.k_scale, seen.v_scale) == (0.5, 0.25) and (c.k_scale, c.v_scale) == (0.5, 0.25)
    pages = Claimed(torch.zeros((5, 16, 2, 64), dtype=torch.bfloat16))
    c.v_pages = pages
    assert seen.v == pages.data_ptr() and seen.k == c.k_pages.data_ptr() != seen.v


def test_assignments_that_do_not_fit_are_refused_and_change_nothing():
    c = claimed_cache()
    before = bytes(c._struct)
    for name, value in (("lens", Claimed(torch.ones(4, dtype=torch.int32))), ("lens", Claimed(torch.ones(3))),
                        ("lens", torch.ones(3, dtype=torch.int32)),  # on the host
                        ("block_table", Claimed(torch.zeros((4, 4), dtype=torch.int32))),
                        ("k_pages", Claimed(torch.zeros((6, 16, 2, 64), dtype=torch.bfloat16))),
                        ("v_pages", Claimed(torch.zeros((5, 16, 2, 64), dtype=torch.float16)))):
        held = getattr(c, name)
        with pytest.raises(ValueError):
            setattr(c, name, value)
        assert getattr(c, name) is held and bytes(c._struct) == before
    with pytest.raises((TypeError, ValueError)):
        c.k_scale = "none"
    assert bytes(c._struct) == before


def test_a_cache_lies_on_one_device():
    def parts():
        return [Claimed(torch.zeros((5, 16, 2, 64), dtype=torch.bfloat16)) for _ in range(2)] + [
            Claimed(torch.zeros((3, 4), dtype=torch.int32)), Claimed(torch.zeros(3, dtype=torch.int32))]
    for i in range(4):
        p = parts()
        p[i] = Claimed(p[i]._t, 1)
        with pytest.raises(ValueError):
            binding.PagedCache(*p)
    c = binding.PagedCache(*parts())
    with pytest.raises(ValueError):
        c.lens = Claimed(torch.zeros(3, dtype=torch.int32), 1)


def elsewhere(good, names, call):
    """call(**good) with each of the named tensors on another GPU, or on the host, in turn."""
    for name in names:
        for t in (Claimed(good[name]._t, 1), good[name]._t):
            with pytest.raises(ValueError):
                call(**{**good, name: t})


class NoLaunch:
    """Stands for the library: a call that gets there has not been refused."""

    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


def test_tensors_on_another_device_than_the_cache_are_refused(monkeypatch):
    c, bf, i32 = claimed_cache(), torch.bfloat16, torch.int32
    monkeypatch.setattr(binding, "_lib", NoLaunch())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    new = dict(k=Claimed(torch.zeros((3, 2, 2, 64), dtype=bf)), v=Claimed(torch.zeros((3, 2, 2, 64), dtype=bf)),
               q=Claimed(torch.zeros((3, 2, 4, 64), dtype=bf)), q_out=Claimed(torch.zeros((3, 2, 4, 64), dtype=bf)),
               inv_freq=Claimed(torch.zeros(8, dtype=torch.float64)), counts=Claimed(torch.zeros(3, dtype=i32)))
    elsewhere(new, list(new), lambda **kw: binding.kda_cache_append(cache=c, **kw))
    packed = dict(k=Claimed(torch.zeros((6, 2, 64), dtype=bf)), v=Claimed(torch.zeros((6, 2, 64), dtype=bf)),
                  cu_seqlens=Claimed(torch.zeros(4, dtype=i32)))
    elsewhere(packed, list(packed), lambda **kw: binding.kda_cache_append(cache=c, **kw))
    monkeypatch.setattr(binding, "_attend_workspace", lambda *a: 0)
    rows = dict(q=Claimed(torch.zeros((3, 2, 4, 64), dtype=bf)), out=Claimed(torch.zeros((3, 2, 4, 64), dtype=bf)),
                counts=Claimed(torch.zeros(3, dtype=i32)))
    elsewhere(rows, list(rows), lambda **kw: binding.kda_cache_attend(cache=c, **kw))
    drafts = dict(draft_tokens=Claimed(torch.zeros((2, 3), dtype=i32)), draft_probs=Claimed(torch.zeros((2, 3, 9))),
                  target_probs=Claimed(torch.zeros((2, 4, 9))), uniform=Claimed(torch.zeros((2, 4))),
                  draft_lens=Claimed(torch.zeros(2, dtype=i32)), counts=Claimed(torch.zeros(2, dtype=i32)),
                  tokens=Claimed(torch.zeros((2, 4), dtype=i32)))
    elsewhere(drafts, list(drafts), binding.kda_draft_accept)


@pytest.mark.parametrize("value,given", [(5, 5), (1 << 31, (1 << 31) - 1), ((1 << 32) + 5, (1 << 31) - 1),
                                         (-1, -1), (-(1 << 32), -1), (-(1 << 32) + 5, -1)])
def test_windows_and_bounds_past_32_bits_are_not_cut_to_their_lower_bits(monkeypatch, value, given):
    """No length passes 2^30, so a larger window or bound is the same as 2^31 - 1."""
    class Library:
        def kda_cache_attend(self, *args):
            self.window, self.max_len = args[10], args[11]
            return 0
    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(binding, "_attend_workspace", lambda *a: 0)
    monkeypatch.setattr(binding, "_stream_of", lambda *a: 0)
    q, out = (Claimed(torch.zeros((3, 2, 4, 64), dtype=torch.bfloat16)) for _ in range(2))
    binding.kda_cache_attend(q, claimed_cache(), out=out, window=value, max_len=value)
    assert (binding._lib.window, binding._lib.max_len) == (given, given)


def test_calls_away_from_the_current_device_or_the_streams_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        binding._stream_of(None, 0)

    class Stream:
        device_index, cuda_stream = 1, 7
    assert binding._stream_of(Stream, 1) == 7
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        binding._stream_of(Stream, 0)


@pytest.mark.gpu
def test_a_cache_follows_lens_that_are_assigned(cuda_device):
    build.build()
    d, bf = 64, torch.bfloat16
    pages = [torch.zeros((2, 16, 1, d), dtype=bf, device="cuda") for _ in range(2)]
    c = binding.PagedCache(*pages, torch.tensor([[1]], dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda())
    k = torch.ones((1, 1, 1, d), dtype=bf, device="cuda")
    c.lens = c.lens + 2
    binding.kda_cache_append(k, k, c)
    c.lens += 4  # in place, and assigned
    binding.kda_cache_append(k, k, c)
    assert pages[0][1, :, 0, 0].nonzero().flatten().tolist() == [5, 9]


@pytest.mark.gpu
def test_tensors_that_do_not_fit_are_refused(cuda_device):
    build.build()
    bf, i32, dev = torch.bfloat16, torch.int32, "cuda"
    pages = torch.zeros((2, 16, 2, 64), dtype=bf, device=dev)
    table, lens = torch.zeros((3, 1), dtype=i32, device=dev), torch.zeros(3, dtype=i32, device=dev)
    for k, v, t, n in ((pages.float(), pages.float(), table, lens), (pages, pages[:1], table, lens),
                       (pages, pages.half(), table, lens), (pages[..., ::2], pages[..., ::2], table, lens),
                       (pages, pages, table.long(), lens), (pages, pages, table, lens[:2]),
                       (pages, pages.transpose(0, 1), table, lens), (pages[0], pages[0], table, lens)):
        with pytest.raises(ValueError):
            binding.PagedCache(k, v, t, n)
    c = binding.PagedCache(pages, pages.clone(), table, lens)
    q = torch.zeros((3, 2, 4, 64), dtype=bf, device=dev)
    k = torch.zeros((3, 2, 2, 64), dtype=bf, device=dev)
    for bad in (q[:2], q[..., :32], q.float().double(), q.transpose(1, 2), q[0], q.cpu(), q[:, ::2].repeat(1, 2, 1, 1)[:, ::2].expand(3, 2, 4, 64)[:, :, ::2]):
        with pytest.raises((ValueError, binding.KDAError)):
            binding.kda_cache_attend(bad, c)
    with pytest.raises(ValueError):
        binding.kda_cache_attend(q, c, counts=torch.zeros(2, dtype=i32, device=dev))
    with pytest.raises(ValueError):
        binding.kda_cache_attend(q, c, out=torch.empty((3, 2, 4, 32), dtype=bf, device=dev))
    with pytest.raises(binding.KDAError):
        binding.kda_cache_attend(q.half(), c)  # a 16-bit cache has the type of the queries
    for args, kw in (((k[:2], k[:2], c), {}), ((k, k[:, :1], c), {}), ((k[:, :, :1], k[:, :, :1], c), {}),
                     ((k, k, c), dict(q=q[:, :1])), ((k, k, c), dict(q_out=q)), ((k, k, c), dict(q=q.half())),
                     ((k, k, c), dict(inv_freq=torch.zeros(32, device=dev))),
                     ((k, k, c), dict(cu_seqlens=torch.zeros(4, dtype=i32, device=dev))),
                     ((k.flatten(0, 1), k.flatten(0, 1), c), dict(cu_seqlens=torch.zeros(3, dtype=i32, device=dev))),
                     ((k, k.cpu(), c), {})):
        with pytest.raises((ValueError, binding.KDAError)):
            binding.kda_cache_append(*args, **kw)
    p = torch.zeros((2, 3, 10), device=dev)
    toks, u = torch.zeros((2, 2), dtype=i32, device=dev), torch.zeros((2, 3), device=dev)
    for args in ((toks[:1], None, p, u), (toks, p, p, u), (toks, None, p, u[:, :2]), (toks.long(), None, p, u),
                 (toks, p[:, :2].half(), p, u), (toks, None, p.transpose(1, 2)[:, :3], u), (toks, None, p.double(), u)):
        with pytest.raises((ValueError, binding.KDAError)):
            binding.kda_draft_accept(*args)
