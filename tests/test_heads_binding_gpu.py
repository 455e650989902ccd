"""What the Python side of the operators on heads promises its callers: workspaces of the stated size, caches whose
tensors move, gradients through autograd, results that other threads and streams do not disturb."""
import pytest
import torch

from reduction_rdx_sum_gb300 import abi

from test_heads_gpu import BF16, DEV, F32, attend_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("q_heads,k_heads,dim", [(32, 8, 128), (10, 2, 80), (4, 4, 64), (4, 2, 256), (24, 2, 112)])
def test_attend_workspace_of_the_stated_size(q_heads, k_heads, dim, dtype):
    q, cache, table, n = attend_case([70, 0, 33, 1], q_heads, k_heads, dim, 16, "int8", dtype)
    want = abi.rdx_kv_attend(q, cache, table, n)
    most = table.shape[1] * 16
    for stated in (abi.rdx_kv_attend_workspace_bytes(cache, 4, q_heads, most, dtype=dtype),
                   abi.rdx_kv_attend_workspace_bytes(cache, 4, q_heads, most)):
        workspace = torch.empty(stated, dtype=torch.uint8, device=DEV)
        assert torch.equal(abi.rdx_kv_attend(q, cache, table, n, workspace=workspace), want)
