"""Edges of the linear attention's calls that the tests beside this one leave out."""
import pytest
import torch

import linear_attention_recurrence_fwd_gb300 as kda
from linear_attention_recurrence_fwd_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("la_type,dtype", [(binding.KDA_BF16, torch.bfloat16), (binding.KDA_F32, torch.float32)])
def test_the_gradient_of_fixed_decays_of_no_sequence_is_zero(la_type, dtype):
    H, d = 5, 64
    around = torch.full((H + 2,), 7.0, dtype=dtype, device="cuda")
    decays = torch.zeros(H, dtype=dtype, device="cuda")
    code = binding.load().kda_linear_bwd(
        None, None, None, None, H * d, H * d, H * d, H * d, decays.data_ptr(), la_type, 0, 1, None, None, None, None, None, None,
        around[1:].data_ptr(), 1, None, 0, 0, H, d, d, 1.0, None, 0, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    assert around.tolist() == [7.0] + [0.0] * H + [7.0]


def test_the_gradient_of_an_empty_batch():
    z = torch.empty((0, 9, 5, 64), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    for x, offsets in ((z, None), (z.flatten(0, 1), cu)):
        g = kda.kda_linear_bwd(x, x, x, torch.zeros(5, device="cuda"), x, cu_seqlens=offsets)
        assert g["q"].shape == x.shape and g["initial_state"].shape == (0, 5, 64, 64)
        assert g["log_alpha"].tolist() == [0.0] * 5
    assert kda.kda_last_device_status() == 0


@pytest.mark.parametrize("rows", [40, 3000])
def test_gradients_where_offsets_leave_no_rows(rows):
    """Offsets that are not allowed (they end before the last row): flagged, and what does not depend on rows is there."""
    H, d = 2, 128
    x = [torch.randn((rows, H, d), device="cuda").to(torch.bfloat16) for _ in range(4)]
    d_final = torch.randn((2, H, d, d), device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    for _ in range(20):
        g = kda.kda_linear_bwd(*x[:3], torch.full((H,), -0.1, device="cuda"), x[3], d_final_state=d_final, cu_seqlens=cu)
        assert torch.equal(g["initial_state"], d_final) and g["log_alpha"].tolist() == [0.0] * H
    assert kda.kda_last_device_status() == 1


def packed(lens, H, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn((sum(lens), H, d), generator=g).to(torch.bfloat16).cuda() for _ in range(4)]
    la = (-0.1 * torch.rand((sum(lens), H), generator=g)).cuda()
    state = torch.randn((len(lens), H, d, d), generator=g).cuda()
    return x, la, state, torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


def test_a_captured_packed_call_follows_its_offsets():
    x, la, state, cu = packed([700, 3, 2000, 0, 297], 2, 128, 91)
    graph = torch.cuda.CUDAGraph()
    call = lambda: (*kda.kda_linear_fwd(*x[:3], la, initial_state=state, cu_seqlens=cu, scale=0.1),  # noqa: E731
                    *kda.kda_linear_bwd(*x[:3], la, x[3], initial_state=state, cu_seqlens=cu, scale=0.1).values())
    call()
    with torch.cuda.graph(graph):
        held = call()
    for lens in ([3000, 0, 0, 0, 0], [0, 1, 1, 2997, 1], [600] * 5, [128, 512, 1024, 1280, 56]):
        cu.copy_(torch.tensor([0] + lens).cumsum(0))
        graph.replay()
        for a, b in zip(call(), held):
            assert torch.equal(a, b), lens
    assert kda.kda_last_device_status() == 0


def test_calls_side_by_side_on_streams():
    """Each call has its workspace; results are those of the calls one after the other."""
    cases = [packed([1900, 40, 1100], 3, 128, 92), packed([5, 0, 1500], 2, 64, 93), packed([300] * 9, 2, 128, 94)]
    call = lambda c, **kw: (*kda.kda_linear_fwd(*c[0][:3], c[1], initial_state=c[2], cu_seqlens=c[3], **kw),  # noqa: E731
                            *kda.kda_linear_bwd(*c[0][:3], c[1], c[0][3], initial_state=c[2], cu_seqlens=c[3], **kw).values())
    want = [call(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [call(c, stream=s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for a, b in zip(w, g):
                assert torch.equal(a, b)
    assert kda.kda_last_device_status() == 0


def test_rows_behind_a_packed_batch_stay():
    """A call on the first rows of larger tensors writes nothing behind them."""
    x, la, state, cu = packed([100, 39], 2, 128, 95)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((200, 2, 128), 7.0, dtype=dtype, device="cuda")
        kda.kda_linear_fwd(*x[:3], la, initial_state=state, cu_seqlens=cu, out=out[:139])
        assert (out[139:] == 7).all() and torch.equal(out[:139], kda.kda_linear_fwd(*x[:3], la, initial_state=state, cu_seqlens=cu,
                                                                                      out_dtype=dtype)[0])
