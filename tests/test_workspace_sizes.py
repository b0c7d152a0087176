"""Sizes of the workspaces a caller brings to the layer norm's backward and to Newton-Schulz (the last test needs a GPU)."""
import pytest
import torch

import grouped_gemm_permute_amd as gg
from grouped_gemm_permute_amd import _lib as L


@pytest.mark.parametrize("T,D", [(0, 64), (1, 64), (512, 1001), (513, 1001), (1024, 768), (1025, 768), (1 << 20, 768), (2000, 16384)])
def test_layer_norm_backward_workspace_size_is_the_entry_points(T, D):
    for dt, enum in ((torch.bfloat16, L.MOE_BF16), (torch.float32, L.MOE_F32)):
        assert gg.layer_norm_backward_workspace_size(T, D, dt) == L.lib().moe_layer_norm_backward_workspace_size(T, D, enum)
    assert gg.layer_norm_backward_workspace_size(1025, 768, torch.bfloat16) > 0
    with pytest.raises(TypeError, match="dtype"):
        gg.layer_norm_backward_workspace_size(T, D, torch.float16)


def test_newton_schulz_workspace_size_of_what_is_not_supported():
    """0, as for sizes out of range, where the matrices' 128 x 128 tiles are 2^24 or more; one tile fewer has a size."""
    size = gg.newton_schulz_workspace_size
    assert size(65535, 4096, 4096) == 0 and size(16384, 4096, 4096) == 0
    assert size(16383, 4096, 4096) > 16383 * 12 * 4096 * 4096
    assert size(65535, 32768, 8) > 0                       # no tiles: short sides of up to 32 have none
    assert size(1, 32769, 64) == 0 and size(65536, 64, 64) == 0
    with pytest.raises(ValueError, match="GPU"):
        gg.newton_schulz(torch.empty(16384, 4096, 4096, device="meta"))


@pytest.mark.gpu
def test_a_callers_workspace_of_just_that_size():
    for T, D, dt in ((1300, 768, torch.bfloat16), (700, 1001, torch.float32), (1100, 9000, torch.bfloat16)):
        x, dy = torch.randn(T, D, device="cuda").to(dt), torch.randn(T, D, device="cuda").to(dt)
        w = torch.ones(D, dtype=dt, device="cuda")
        f = gg.layer_norm(x, w)
        want = gg.layer_norm_backward(x, dy, f["rstd"], f["mean"], w, bias_grad=True)
        need = gg.layer_norm_backward_workspace_size(T, D, dt)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")      # NaN patterns
        for _ in range(2):
            got = gg.layer_norm_backward(x, dy, f["rstd"], f["mean"], w, bias_grad=True, workspace=ws)
            assert all(torch.equal(got[k], want[k]) for k in ("dx", "dweight", "dbias"))
        with pytest.raises(ValueError, match="needs"):
            gg.layer_norm_backward(x, dy, f["rstd"], f["mean"], w, bias_grad=True, workspace=ws[:-1])


@pytest.mark.gpu
def test_matrices_without_rows_or_columns_are_refused_as_such():
    for shape in ((2, 0, 5), (2, 5, 0), (0, 0)):
        W, m = torch.empty(shape, device="cuda"), torch.empty(shape, device="cuda")
        for call in (lambda: gg.newton_schulz(W), lambda: gg.muon_step(W, m, m, 0.1)):
            with pytest.raises(gg.MoeError, match="INVALID_ARG"):
                call()
