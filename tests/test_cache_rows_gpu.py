"""Cache writing and reading at the sizes of prompts, where a group of threads takes four heads, against the definition:
codes and scales bit for bit, with some slots outside the cache."""
import numpy as np
import pytest
import torch

from oracle import heads
from reduction_rdx_sum_gb300 import abi

from test_heads_gpu import BF16, DEV, F32, FORMATS, host, make_rows, seeded, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["plain", "slice", "heads", "off"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("shape", [
    # tokens, heads, head_dim, page: more blocks of one head each than four for each SM; heads left over from groups of four
    (3001, 8, 128, 64), (4099, 5, 80, 48), (40000, 1, 64, 16), (2500, 7, 256, 33), (13001, 12, 16, 16), (9001, 3, 48, 100),
], ids=str)
def test_prompts(shape, fmt, dtype, layout):
    tokens, n_heads, dim, page = shape
    g = seeded(tokens)
    k, v = make_rows(g, tokens, n_heads, dim, dtype, layout), make_rows(g, tokens, n_heads, dim, dtype, layout)
    v[tokens // 2, n_heads - 1, 3] = float("inf")
    k[tokens - 1, n_heads - 1, 1] = float("nan")
    pages = -(-tokens // page) + 2
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:tokens]
    slots[7::500] = -1
    slots[11::700] = pages * page + 5
    at = slots.cpu().numpy()
    inside = (at >= 0) & (at < pages * page)
    cache = abi.KVCache.zeros(pages, page, n_heads, dim, FORMATS[fmt], DEV)
    abi.rdx_kv_write(cache, k, v, slots)
    want = {}
    for name, x, codes, scale in (("k", k, cache.k, cache.k_scale), ("v", v, cache.v, cache.v_scale)):
        c, s = heads.quantise(host(x), fmt)
        full = np.zeros((pages, n_heads, page, dim))
        full[at[inside] // page, :, at[inside] % page] = c[inside]
        assert np.array_equal(values(codes), full)
        full = np.zeros((pages, n_heads, page), np.float32)
        full[at[inside] // page, :, at[inside] % page] = s[inside]
        assert np.array_equal(host(scale), full, equal_nan=True)
        want[name] = c.astype(np.float32) * s[..., None]
        want[name][at < 0] = 0
        want[name][at >= pages * page] = np.nan
    out = [make_rows(g, tokens, n_heads, dim, dtype, layout) for _ in range(2)]
    abi.rdx_kv_read(cache, slots, dtype=dtype, k_out=out[0], v_out=out[1])
    for name, y in zip("kv", out):
        ref = torch.from_numpy(want[name]).to(dtype).to(DEV)
        assert torch.equal(y.isnan(), ref.isnan()) and torch.equal(y.nan_to_num(nan=0.0), ref.nan_to_num(nan=0.0))
