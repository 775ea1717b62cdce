"""Corners of the expert operators' binding that need no GPU."""
import pytest

torch = pytest.importorskip("torch")
import torch.autograd.forward_ad as fwd  # noqa: E402

from differentiable_soft_top_b200 import experts as ex  # noqa: E402


def test_a_forward_mode_tangent_counts_as_tracked():
    """A dual tensor does not require grad; without this the tangent would be lost in the direct path."""
    x, y = torch.randn(3), torch.randn(3)
    with fwd.dual_level():
        d = fwd.make_dual(x, torch.ones(3))
        assert ex._tracked(None, d) and not ex._tracked(x, None, y)
        with torch.no_grad():  # no_grad does not switch forward mode off
            assert ex._tracked(y, d)
    assert not ex._tracked(x) and ex._tracked(x, y.requires_grad_())
