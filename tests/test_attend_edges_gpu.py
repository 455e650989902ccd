"""Attention over the cache at the ends of its ranges: lengths near 2^31, weights that nearly cancel, bfloat16 rows off
their alignment.  References in float64; each tolerance is derived where it stands."""
import math

import pytest
import torch

from reduction_rdx_sum_gb300 import abi

from test_heads_gpu import DEV, F32, FORMATS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dim", [16, 144])
def test_lengths_up_to_the_last(dim, fmt):
    # one page of 2^18 tokens named 2^13 times; every score is the same, far below 0, and every value row: one place past
    # the end that kept its score of 0 would outweigh all the others.  A warp adds the 4 weights a lane has of each of its
    # pieces (2^31 tokens in pieces of 16 at least, over 1216 warps at least), each addition rounded: 2^19 2^-24 for the
    # sum, as much for the weighted ones.
    page = 1 << 18
    cache = abi.KVCache.zeros(1, page, 1, dim, FORMATS[fmt], DEV)
    value = torch.linspace(-2, 2, dim, device=DEV)
    rows = torch.ones(page, 1, dim, device=DEV)
    abi.rdx_kv_write(cache, rows, value.expand(page, 1, dim), torch.arange(page, device=DEV))
    _, v = abi.rdx_kv_read(cache, torch.zeros(1, dtype=torch.int64, device=DEV), dtype=F32)
    table = torch.zeros(1, 1 << 13, dtype=torch.int32, device=DEV)
    q = torch.full((1, 1, dim), -1.0, device=DEV)
    bound = 2.0 ** (19 - 24)
    for n in (2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 17, 2 ** 31 - 31, 2 ** 31 - 33):
        for score in (20.0, 80.0):
            lse = torch.zeros(1, 1, device=DEV)
            lens = torch.tensor([n], dtype=torch.int32, device=DEV)
            out = abi.rdx_kv_attend(q, cache, table, lens, scale=score / dim, max_len=2 ** 31 - 1, lse=lse)
            assert bool(((out - v).abs() <= 2 * bound * v.abs() + 1e-6).all()), (n, score)
            assert abs(lse.item() - (math.log(n) - score)) <= 1.5 * bound, (n, score)
