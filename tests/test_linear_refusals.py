"""What the linear attention's and the logits' C calls refuse, before anything is launched (no GPU)."""
import ctypes

import pytest

from linear_attention_recurrence_fwd_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


F, MIS, ODD = ctypes.c_void_p(16), ctypes.c_void_p(24), ctypes.c_void_p(17)


def fwd(lib, q=F, k=F, v=F, qs=256, ks=256, vs=256, la=F, la_type=0, lt=2, lh=1, cu=None, s0=None, out=F, dt=1, s1=None,
        N=1, T=8, H=2, dk=128, dv=128, ws=None, need=0):
    return lib.kda_linear_fwd(q, k, v, qs, ks, vs, la, la_type, lt, lh, cu, s0, out, dt, s1, N, T, H, dk, dv, 1.0, ws, need, None)


def bwd(lib, do=F, dos=256, dq=F, dla=F, ds0=None, d1=None, N=1, T=8, la=F, dk=128):
    return lib.kda_linear_bwd(F, F, F, do, 256, 256, 256, dos, la, 0, 2, 1, None, None, d1, dq, F, F, dla, 0, ds0, N, T, 2, dk, dk,
                              1.0, None, 0, None)


BAD = [(dict(q=None), 1), (dict(k=None), 1), (dict(la=None), 1), (dict(out=None), 1), (dict(N=-1), 1), (dict(T=-1), 1),
       (dict(H=0), 1), (dict(N=3), 1), (dict(N=0), 1), (dict(qs=-8), 1), (dict(lt=-1), 1), (dict(dk=96, dv=96), 2),
       (dict(dk=128, dv=64), 2), (dict(dt=2), 2), (dict(dt=3), 2), (dict(la_type=2), 2), (dict(T=1 << 30, H=1 << 16), 2),
       (dict(H=(1 << 16) + 1), 2), (dict(q=MIS), 3), (dict(v=MIS), 3), (dict(qs=257), 3), (dict(vs=4), 3), (dict(la=ODD), 3),
       (dict(la=ctypes.c_void_p(18), la_type=1), 3), (dict(s0=MIS), 3), (dict(s1=MIS), 3), (dict(out=MIS), 3),
       (dict(cu=ctypes.c_void_p(18)), 3)]


@pytest.mark.parametrize("args,code", BAD)
def test_forward(lib, args, code):
    assert fwd(lib, **args) == code


@pytest.mark.parametrize("args,code", [(dict(do=None), 1), (dict(dq=None), 1), (dict(N=3), 1), (dict(dos=-1), 1), (dict(dk=32), 2),
                                       (dict(do=MIS), 3), (dict(dos=12), 3), (dict(dq=MIS), 3), (dict(dla=ODD), 3),
                                       (dict(ds0=MIS), 3), (dict(d1=MIS), 3)])
def test_backward(lib, args, code):
    assert bwd(lib, **args) == code


@pytest.mark.parametrize("name", ["qs", "ks", "vs"])
def test_rows_that_overlap_or_lie_too_far_apart(lib, name):
    # one tensor map holds an operand's rows: 2^40 bytes between two at most
    assert fwd(lib, **{name: 248}) == fwd(lib, **{name: 0}) == 1
    assert fwd(lib, **{name: 1 << 38}) == 2


def test_gradient_rows_that_overlap_or_lie_too_far_apart(lib):
    assert bwd(lib, dos=248) == bwd(lib, dos=0) == 1
    assert bwd(lib, dos=1 << 38) == 2


def test_nothing_to_do_and_workspaces(lib):
    assert fwd(lib, N=0, T=0, q=None, k=None, v=None, la=None, out=None) == 0
    assert lib.kda_linear_fwd_workspace_size(0, 10, 2, 128, 128, 0) == 0
    assert lib.kda_linear_fwd_workspace_size(1, 10, 2, 96, 96, 0) == 0
    assert lib.kda_linear_bwd_workspace_size(1, 0, 2, 128, 128, 1) == 0


def test_tokens(lib):
    step = lambda q=F, s=F, out=F, N=4, d=128, la=F, dt=1: lib.kda_linear_step(  # noqa: E731
        q, F, F, 256, 256, 256, la, 0, 2, 1, s, out, dt, N, 2, d, d, 1.0, None)
    assert step(q=None) == step(s=None) == step(out=None) == step(N=-1) == 1
    assert step(d=32) == step(dt=2) == 2
    assert step(q=MIS) == step(s=MIS) == step(out=MIS) == step(la=ODD) == 3
    assert step(N=0) == 0
    verify = lambda s=F, out=F, K=4: lib.kda_linear_verify(F, F, F, 256, 256, 256, F, 0, 2, 1, s, out, 1, 3, K, 2, 128, 128, 1.0, None)  # noqa: E731
    assert verify(s=None) == verify(out=None) == verify(K=-1) == 1
    assert verify(K=0) == 0
    commit = lambda acc=F, K=4: lib.kda_linear_commit(F, F, 256, 256, F, 0, 2, 1, F, acc, 3, K, 2, 128, 128, None)  # noqa: E731
    assert commit(acc=None) == commit(K=-2) == 1
    assert commit(K=0) == 0


def test_logits(lib):
    def call(x=F, dt=1, sn=100, sr=100, out=F, odt=1, N=1, R=1, V=100, **rules):
        u = binding._LogitsRules(**rules)
        return lib.kda_logits_probs(x, dt, sn, sr, ctypes.addressof(u), out, odt, N, R, V, None)
    assert call(x=None) == call(out=None) == call(N=-1) == call(R=-1) == call(V=0) == call(sn=-1) == 1
    assert call(L=-1) == call(J=-1) == call(tokens_stride=-1) == call(mask_stride_n=-1) == call(J=2, bias=16) == 1
    assert call(dt=3) == call(odt=0) == call(dt=0, odt=2) == call(V=(1 << 30) + 1) == 2
    assert call(V=409601, presence=16) == call(N=1 << 20, R=1 << 10) == 2
    assert call(x=ctypes.c_void_p(18)) == call(dt=0, x=ODD) == call(tokens=18) == call(temperature=17) == call(out=ODD) == 3
    assert call(N=0) == call(R=0) == 0
