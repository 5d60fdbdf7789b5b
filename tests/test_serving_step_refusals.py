"""What the example's block refuses, without a GPU: the check runs ahead of anything else."""
import pytest

from tests.test_gpu_serving_step import _example


@pytest.mark.parametrize("window,sinks", [(40, 0), (40, 4)])
def test_chosen_pages_have_no_window(window, sinks):
    block = _example().Block
    with pytest.raises(ValueError):
        block.__call__(None, None, None, None, window=window, sinks=sinks, blocks=8)
