"""More sizes, layouts and far values of the operators of a trainable expert block
(MI355X); forms and tolerances as in test_train_gpu.py."""
import pytest

from tests import test_train_gpu as base
from tests.test_train_gpu import BF, F32, moe  # noqa: F401

pytestmark = pytest.mark.gpu


# (rows of more than 8192 columns: the borders of the row workgroups and of one launch)
@pytest.mark.parametrize("T,H", [(64, 8200), (320, 10001), (321, 10001), (512, 12288), (513, 12288), (1000, 16384), (1024, 8201), (1025, 8200)])
@pytest.mark.parametrize("kind", [(BF, True), (F32, False)])
def test_layer_norm_backward_of_wide_rows(moe, T, H, kind):  # noqa: F811
    base.test_layer_norm_backward(moe, T, H, kind)
