"""The kernels' bounded waits, in forms that fault and hang nothing (-m gpu): a wait that runs out gives the whole
warp one answer, raises the device error word and leaves the context usable."""

import pytest
import torch

from compressed_kv_sparse_compressor_gb300 import abi
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    abi.check(abi.ds4c_test_set_wait_limit(0), "ds4c_test_set_wait_limit")


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("kernels", [abi.DS4C_WAITS_QUANT_MATMUL])
def test_lanes_that_see_different_things_get_one_answer(kernels):
    """Half of the lanes find their barrier complete, the others' wait runs out: no lane may go on alone."""
    answers = torch.full((96,), -7, dtype=torch.int32, device="cuda")
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    assert abi.ds4c_test_set_wait_limit(20000) == abi.DS4C_OK                  # 20 us
    try:
        assert abi.ds4c_test_warp_wait(kernels, answers.data_ptr(), stream()) == abi.DS4C_OK
        assert abi.ds4c_sync_status(stream()) == abi.DS4C_ERR_DEVICE
    finally:
        assert abi.ds4c_test_set_wait_limit(0) == abi.DS4C_OK
    assert abi.ds4c_sync_status(stream()) == abi.DS4C_OK
    assert answers.tolist() == [0] * 64 + [1] * 32
