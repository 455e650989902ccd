"""Attention over the cache at the ends of its ranges: lengths near 2^31, weights that nearly cancel, bfloat16 rows off
their alignment.  References in float64; each tolerance is derived where it stands."""
import math

import pytest
import torch

from reduction_rdx_sum_gb300 import abi

from test_heads_gpu import BF16, DEV, F32, FORMATS, attend_case, check_attend, make_rows, seeded

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


def both_ways(table, page, longest):
    """A close bound, which takes few and short sequences through clusters, and a wide one with its wide table."""
    wide = torch.full((table.shape[0], 1 + 200000 // page), -5, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    return (table, longest), (wide, 200000)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_weights_that_nearly_cancel(dim, fmt):
    # two tokens with opposite codes and scales that differ by up to 2^-13: a bfloat16 result of 2^-13 of the values shows
    # what its weights' roundings leave.  Scores below 1/4: ds as in test_heads_gpu.py, (dim / 8 + 16) 2^-23 / 4, twice;
    # weights of 24 bits and an exponential to two units in the last place: 2^-23 + 2^-22; 16 products and the joined
    # sums 2^-22.  Weights of 16 bits would be off by up to 2^-17.
    g = seeded(dim)
    batch, hq, hk = 40, 8, 2
    cache = abi.KVCache.zeros(batch, 16, hk, dim, FORMATS[fmt], DEV)
    codes = torch.randint(1, 120, (batch, hk, 1, dim), generator=g, device=DEV).to(FORMATS[fmt])
    cache.v[:, :, :1].view(torch.int8).copy_(codes.view(torch.int8))
    cache.v[:, :, 1:2].copy_(-codes.float())
    cache.v_scale[:, :, 0] = 1 + torch.rand(batch, hk, generator=g, device=DEV)
    cache.v_scale[:, :, 1] = cache.v_scale[:, :, 0] * (1 + 2.0 ** -13 * torch.rand(batch, hk, generator=g, device=DEV))
    k = torch.randn(batch, hk, 2, dim, generator=g, device=DEV)
    top = 127 if fmt == "int8" else 448
    cache.k[:, :, :2].copy_((k * top / 8).round().clamp(-top, top))
    cache.k_scale.fill_(8 / top)
    q = torch.randn(batch, hq, dim, generator=g, device=DEV).bfloat16()
    kd = cache.k[:, :, :2].double() * cache.k_scale[:, :, :2, None].double()
    vd = cache.v[:, :, :2].double() * cache.v_scale[:, :, :2, None].double()
    qd = q.double().view(batch, hk, hq // hk, dim)
    size = (qd.abs() @ kd.abs().transpose(-1, -2)).max()
    scale = float(0.25 / size)
    ref = (torch.softmax(scale * qd @ kd.transpose(-1, -2), -1) @ vd).view(batch, hq, dim)
    ds = (dim / 8 + 16) * 2.0 ** -23 / 4
    unit = 2 * ds + 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -22
    bound = vd.abs().amax(2).repeat_interleave(hq // hk, 1) * unit + 2.0 ** -8 * ref.abs()
    table = torch.arange(batch, dtype=torch.int32, device=DEV)[:, None]
    lens = torch.full((batch,), 2, dtype=torch.int32, device=DEV)
    for wide, longest in both_ways(table, 16, 2):
        out = abi.rdx_kv_attend(q, cache, wide, lens, scale=scale, max_len=longest)
        off = (out.double() - ref).abs() / bound
        assert float(off.max()) <= 1, (longest, float(off.max()))


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_sums_that_grow_and_cancel(fmt):
    # ten million tokens, pages of 2048 in turn of a value row and of its opposite, all scores equal: the sums of a run
    # grow over one page and cancel over the next, and the result is 0.  Roundings to the nearest of A additions in each
    # of W runs leave at most sqrt(A / W) 2^-26 of the values as a standard deviation, 2^-23 at eight of them; sums that
    # lose what each step shifts out, always towards 0, would leave 2^-17 of the values where runs and pages are in step
    # (2432 runs of 128 pieces of 32 tokens, two pieces' worth of each for its start).
    page, dim, hq = 2048, 64, 8
    g = seeded(5)
    cache = abi.KVCache.zeros(2, page, 1, dim, FORMATS[fmt], DEV)
    codes = torch.randint(1, 100, (page, dim), generator=g, device=DEV).float()
    cache.v[0, 0].copy_(codes)
    cache.v[1, 0].copy_(-cache.v[0, 0].float())
    cache.v_scale.copy_((1 + torch.rand(page, generator=g, device=DEV)).expand(2, 1, page))
    cache.k.copy_(torch.ones_like(cache.k, dtype=F32))
    cache.k_scale.fill_(0.25)
    n = (2432 * 128 - 2) * 32
    table = (torch.arange(-(-n // page), device=DEV) % 2).int()[None]
    q = torch.randn(1, hq, dim, generator=g, device=DEV).bfloat16()
    v = cache.v[0, 0].double() * cache.v_scale[0, 0, :, None].double()
    left = n % (2 * page)
    ref = (v[:left] if left <= page else v[left - page:]).sum(0) / n
    out = abi.rdx_kv_attend(q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV))
    bound = 2.0 ** -20 * v.abs().mean(0) + 2.0 ** -8 * ref.abs()
    off = (out[0].double() - ref).abs() / bound
    assert float(off.max()) <= 1, float(off.max())


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("case", [([300, 17, 0], 8, 2, 64, 16), ([90, 200], 12, 1, 128, 48), ([33], 5, 5, 80, 7),
                                  ([77, 1], 6, 2, 256, 32)], ids=str)
def test_bfloat16_rows_of_every_layout(case, fmt):
    # rows read and written value by value, or four at a time, are the same rows
    lens, hq, hk, dim, page = case
    q, cache, table, n = attend_case(lens, hq, hk, dim, page, fmt, BF16)
    for wide, longest in both_ways(table, page, max(lens)):
        lse = torch.empty(len(lens), hq, device=DEV)
        want = abi.rdx_kv_attend(q, cache, wide, n, lse=lse, max_len=longest)
        check_attend(want, lse, q, cache, wide, n, dim ** -0.5, BF16)
        for layout in ("slice", "heads", "off"):
            x = make_rows(seeded(1), len(lens), hq, dim, BF16, layout).copy_(q)
            y = make_rows(seeded(2), len(lens), hq, dim, BF16, layout)
            abi.rdx_kv_attend(x, cache, wide, n, out=y, max_len=longest)
            assert torch.equal(y, want), layout
