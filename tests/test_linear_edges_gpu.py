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
