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


def test_cache_follows_its_tensors():
    # a cache's storage may move between calls: each call goes to where it is, none to where it was
    q, cache, table, n = attend_case([70, 33], 4, 2, 64, 16, "int8", F32)
    want = abi.rdx_kv_attend(q, cache, table, n)
    slots = torch.arange(cache.pages * 16, device=DEV)
    rows = abi.rdx_kv_read(cache, slots, dtype=F32)
    old = [x.data for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    kept = [x.clone() for x in old]
    for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        x.data = x.data.clone()
    assert cache.k.data_ptr() != old[0].data_ptr()
    for x in old:
        x.zero_()
    assert torch.equal(abi.rdx_kv_attend(q, cache, table, n), want)
    new = torch.randn(1, 2, 64, device=DEV)
    abi.rdx_kv_write(cache, new, new, slots[:1])
    assert not any(x.any() for x in old)
    got = abi.rdx_kv_read(cache, slots, dtype=F32)
    for a, b in zip(rows, got):
        assert torch.equal(a[1:].nan_to_num(nan=1e9), b[1:].nan_to_num(nan=1e9))
        assert torch.allclose(b[0], new[0], atol=float(new.abs().max()) / 127)
    # away on the CPU or given back: refused; brought in again: as before
    for x, keep in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), kept):
        here = x.data
        x.data = here.cpu()
        with pytest.raises(TypeError):
            abi.rdx_kv_attend(q, cache, table, n)
        x.data = here
        bytes_ = x.untyped_storage().nbytes()
        x.untyped_storage().resize_(0)
        for call in (lambda: abi.rdx_kv_attend(q, cache, table, n), lambda: abi.rdx_kv_write(cache, new, new, slots[:1]),
                     lambda: abi.rdx_kv_read(cache, slots)):
            with pytest.raises(ValueError):
                call()
        x.untyped_storage().resize_(bytes_)
        x.copy_(keep)
    assert torch.equal(abi.rdx_kv_attend(q, cache, table, n), want)
