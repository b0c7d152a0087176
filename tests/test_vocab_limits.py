"""Cross entropy and distillation at the limits of their sizes, as far as the host decides (no GPU needed; no pointer here is
dereferenced, and no call here has anything to launch)."""
import pytest

from test_vocab_binding import DIST_BACK, LOSS_BACK, UNSUPPORTED, call

ROOM = dict(n=1 << 62)


@pytest.mark.parametrize("name,defaults", [("moe_cross_entropy_backward", LOSS_BACK), ("moe_distillation_backward", DIST_BACK)])
@pytest.mark.parametrize("over", [dict(T=1 << 28, D=257), dict(T=1 << 28, D=512), dict(T=(1 << 22) + 1, D=16384), dict(T=(1 << 27) + 1, D=512)])
def test_a_dh_of_too_many_tiles_is_refused_before_the_first_launch(name, defaults, over):
    assert call(name, defaults, dict(over, **ROOM)) == UNSUPPORTED
    assert call(name, defaults, dict(over, dW=None, **ROOM)) == UNSUPPORTED
