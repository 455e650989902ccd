"""The Python side of the operators on heads, without a GPU: caches of fake CUDA tensors (shapes, types and devices, no
memory) through the checks that come before any CUDA call."""
import ctypes
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from reduction_rdx_sum_gb300 import abi, build

from test_heads_host import Attend, Cache

TYPES = {torch.float32: 0, torch.bfloat16: 1}


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load()


def fake_cache(pages, page, heads, dim, dtype=torch.int8):
    with warnings.catch_warnings(), FakeTensorMode():
        warnings.simplefilter("ignore")  # of reading a fake tensor's address
        return abi.KVCache.zeros(pages, page, heads, dim, dtype, "cuda")


@pytest.mark.parametrize("q_heads,k_heads", [(1, 1), (32, 8), (10, 2), (24, 2), (64, 1)])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 192, 256])
def test_attend_workspace_of_each_type(lib, dim, q_heads, k_heads):
    cache = fake_cache(5, 48, k_heads, dim)
    for batch, max_len in ((1, 1), (8, 100), (300, 48), (3, 100000)):
        need = {}
        for dtype, code in TYPES.items():
            a = Attend(cache=Cache(pages=5, page_size=48, heads=k_heads, head_dim=dim), batch=batch, q_heads=q_heads,
                       table_pages=-(-max_len // 48), max_len=max_len, type=code, scale=1.0)
            need[dtype] = lib.rdx_kv_attend_workspace_bytes(ctypes.byref(a))
            assert need[dtype] > 0
            assert abi.rdx_kv_attend_workspace_bytes(cache, batch, q_heads, max_len, dtype=dtype) == need[dtype]
        # without a type: enough for either
        assert abi.rdx_kv_attend_workspace_bytes(cache, batch, q_heads, max_len) == max(need.values())


def test_attend_workspace_refuses_other_types(lib):
    with pytest.raises(TypeError):
        abi.rdx_kv_attend_workspace_bytes(fake_cache(5, 48, 2, 64), 8, 4, 100, dtype=torch.float16)


@pytest.mark.parametrize("shape", [(4, 0, 2, 64), (4, 16, 0, 64), (4, 16, 2, 0), (0, 0, 2, 64)], ids=str)
def test_caches_without_rows_in_a_page_are_refused(shape):
    # attention divides by page_size; a cache of no pages is one that has no room yet
    with pytest.raises(ValueError):
        fake_cache(*shape)
    assert fake_cache(0, 16, 2, 64).pages == 0


def marshalled(cache):
    """A call's first step, which takes the cache apart; the ones after it need a GPU."""
    abi._marshal().kv_read(cache, None, 0, None, None, None)


def test_cache_tensors_cannot_be_replaced():
    cache = fake_cache(4, 16, 2, 64)
    for name in ("k", "v", "k_scale", "v_scale", "pages", "heads", "page_size", "head_dim"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))
    assert (cache.pages, cache.page_size, cache.heads, cache.head_dim) == (4, 16, 2, 64)


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
def test_caches_without_their_memory_are_refused(name):
    # storage given back (offloading), or smaller than the tensor; a tensor of another shape
    def changes(x):
        yield lambda: x.untyped_storage().resize_(0)
        yield lambda: x.untyped_storage().resize_(x.numel() * x.element_size() - 1)
        yield lambda: x.resize_(3, *x.shape[1:])
        yield lambda: x.transpose_(1, 2)
        yield lambda: x.resize_(0, *x.shape[1:])

    for i in range(5):
        with warnings.catch_warnings(), FakeTensorMode():
            warnings.simplefilter("ignore")
            cache = abi.KVCache.zeros(4, 16, 2, 64, torch.int8, "cuda")
            list(changes(getattr(cache, name)))[i]()
            with pytest.raises((TypeError, ValueError), match=f"KVCache|{name}"):
                marshalled(cache)


@pytest.mark.parametrize("given", ["q_out", "k_out", "cos", "sin"])
def test_gradients_that_nothing_returns_are_refused(given):
    # outputs of the caller's own, and the tables, have no place in autograd: an error, not a lost gradient
    with warnings.catch_warnings(), FakeTensorMode():
        warnings.simplefilter("ignore")
        q, k = torch.empty(3, 2, 64, device="cuda"), torch.empty(3, 1, 64, device="cuda")
        w = torch.empty(64, device="cuda").requires_grad_(given in ("q_out", "k_out"))
        table = {"cos": torch.empty(5, 32, device="cuda"), "sin": torch.empty(5, 32, device="cuda")}
        out = {}
        if given in table:
            table[given].requires_grad_()
        else:
            out[given] = torch.empty_like(q if given == "q_out" else k)
        positions = torch.empty(3, dtype=torch.int64, device="cuda")
        with pytest.raises(RuntimeError, match="rdx_qk_norm_rope: .*gradient"):
            abi.rdx_qk_norm_rope(q, k, w, w, positions, table["cos"], table["sin"], **out)
