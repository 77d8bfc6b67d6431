"""A status word that a fork wrote, read with the call that reads all others."""
import pytest
import torch

import rmsnorm_fp4_quant_gb300 as fq
from rmsnorm_fp4_quant_gb300 import build as fbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    fbuild.build()
    fq.lib()


@pytest.mark.parametrize("read", ["fp4_read_device_status", "fp4_kv_read_status"])
def test_pages_that_run_out_are_read_as_such(read):
    cache = [torch.zeros(1, 1, 16, 32, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, 16, 4, dtype=torch.uint8, device="cuda"),
             torch.zeros(1, 1, 16, 32, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, 4, 16, dtype=torch.uint8, device="cuda")]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")      # noqa: E731
    status = i32([0])
    stream = torch.cuda.current_stream().cuda_stream
    fq.kv_fork_nvfp4(cache, i32([1]), i32([[0, -1]]), i32([15]), status=status)
    assert getattr(fq, read)(status.data_ptr(), stream) == fq.FP4_OK
    fq.kv_fork_nvfp4(cache, i32([1]), i32([[0, -1]]), i32([16]), status=status)
    assert getattr(fq, read)(status.data_ptr(), stream) == fq.FP4_ERR_NO_PAGES
    status.fill_(77)                                         # no status at all
    assert getattr(fq, read)(status.data_ptr(), stream) == fq.FP4_ERR_INVALID_ARG
