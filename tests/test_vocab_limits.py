"""Cross entropy and distillation at the limits of their sizes, as far as the host decides (no GPU needed; no pointer here is
dereferenced, and no call here has anything to launch)."""
import pytest
import torch

from test_vocab_binding import BAD, DIST, DIST_BACK, LOSS_BACK, OK, UNSUPPORTED, call, gg

ROOM = dict(n=1 << 62)


@pytest.mark.parametrize("name,defaults", [("moe_cross_entropy_backward", LOSS_BACK), ("moe_distillation_backward", DIST_BACK)])
@pytest.mark.parametrize("over", [dict(T=1 << 28, D=257), dict(T=1 << 28, D=512), dict(T=(1 << 22) + 1, D=16384), dict(T=(1 << 27) + 1, D=512)])
def test_a_dh_of_too_many_tiles_is_refused_before_the_first_launch(name, defaults, over):
    assert call(name, defaults, dict(over, **ROOM)) == UNSUPPORTED
    assert call(name, defaults, dict(over, dW=None, **ROOM)) == UNSUPPORTED


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D,V", [(64, 8, 1 << 24), (64, 64, 1 << 23), (33, 8, 1 << 24), (128, 8, 1 << 24), (40000, 64, 1 << 20)])
def test_dz_of_a_piece_is_two_gib_at_most(T, D, V, dtype):
    """Beside it: its rows' padding, copies of h and (above 64 rows) of the table in planes, parts of dh."""
    rows = T * 256 * (4 if dtype == torch.bfloat16 else 6)
    copies = 6 * (T + 64) * (D + 128) + (6 * (V + 64) * (D + 128) if T > 64 else 0)
    parts = 2 * 256 * 64 * D * 4 + 512 * 65536 * 4 + 64 * T + T * (D + 32) * 4
    for need in (gg.cross_entropy_workspace_size(T, D, V, dtype, True), gg.distillation_workspace_size(T, D, V, 9, dtype, True)):
        assert 1 << 29 < need <= (2 << 30) + rows + copies + parts


@pytest.mark.parametrize("name,defaults", [("moe_distillation_forward", DIST), ("moe_distillation_backward", DIST_BACK)])
def test_temperatures_whose_log2_of_e_overflows_are_refused(name, defaults):
    """1 / 4e-39 is an fp32 number, log2(e) / 4e-39 is none."""
    none = dict(T=0, h=None, W=None, ids=None, q=None, lse=None, z=None, ws=None, **({"loss": None} if "loss" in defaults else {"g": None, "dh": None, "dW": None}))
    for tau in (4e-39, 3e-39, 3.403e38):
        assert call(name, defaults, dict(none, tau=tau)) == BAD
    for tau in (4.4e-39, 1.0, 3.39e38):
        assert call(name, defaults, dict(none, tau=tau)) == OK
