"""What the Python side of the operators on heads promises its callers: workspaces of the stated size, caches whose
tensors move, gradients through autograd, results that other threads and streams do not disturb."""
import ctypes
import os
import subprocess
import threading

import pytest
import torch

from reduction_rdx_sum_gb300 import abi

from test_heads_gpu import BF16, DEV, F32, attend_case, qk_case, seeded

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


def plain_norm_rope(x, w, pos, cos, sin, interleaved, eps):
    n = x * w / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    rot = 2 * cos.shape[1]
    a, b = (n[..., 0:rot:2], n[..., 1:rot:2]) if interleaved else (n[..., :rot // 2], n[..., rot // 2:rot])
    y = a * c - b * s, b * c + a * s
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, n[..., rot:]), -1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_rope_under_autograd(dtype, interleaved):
    q, k, wq, wk, pos, cos, sin = qk_case(37, 6, 2, 64, 32, dtype, "slice")
    g = seeded(3)
    dq, dk = torch.randn(q.shape, generator=g, device=DEV).to(dtype), torch.randn(k.shape, generator=g, device=DEV).to(dtype)
    want = abi.rdx_qk_norm_rope(q, k, wq, wk, pos, cos, sin, interleaved=interleaved)
    grads = abi.rdx_qk_norm_rope_grad(dq, dk, q, k, wq, wk, pos, cos, sin, interleaved=interleaved)
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, wq, wk)]
    out = abi.rdx_qk_norm_rope(*leaves, pos, cos, sin, interleaved=interleaved)
    assert all(torch.equal(a, b) and a.requires_grad for a, b in zip(out, want))
    torch.autograd.backward(out, (dq, dk))
    for x, grad in zip(leaves, grads):
        assert torch.equal(x.grad, grad)
    # the same from the formula in 64 bits; a float32 kernel's bound is 60 u of absolute terms (see test_heads_gpu.py),
    # far below 2^-12 of the largest of a row's or column's gradients; a bfloat16 result adds half a unit, 2^-8
    exact = [x.detach().double().requires_grad_() for x in (q, k, wq, wk)]
    y = [plain_norm_rope(exact[i], exact[2 + i], pos, cos, sin, interleaved, 1e-6) for i in range(2)]
    torch.autograd.backward(y, (dq.double(), dk.double()))
    for i, (x, ref) in enumerate(zip(leaves, exact)):
        top = ref.grad.abs().amax(-1, keepdim=True)
        assert bool(((x.grad.double() - ref.grad).abs() <= top * (2.0 ** -8 if dtype is BF16 and i < 2 else 2.0 ** -12)).all())


def test_norm_rope_gradients_of_some_arguments():
    q, k, wq, wk, pos, cos, sin = qk_case(9, 4, 2, 64, 64, F32)
    w = wq.clone().requires_grad_()
    a, b = abi.rdx_qk_norm_rope(q, k, w, wk, pos, cos, sin)
    (a.sum() + 2 * b.sum()).backward()  # gradients of one value for all: strides of 0
    ones = torch.ones_like(q), torch.full_like(k, 2)
    assert torch.equal(w.grad, abi.rdx_qk_norm_rope_grad(*ones, q, k, wq, wk, pos, cos, sin)[2])
    # one result unused: its gradient is zeros
    x = q.clone().requires_grad_()
    abi.rdx_qk_norm_rope(x, k, wq, wk, pos, cos, sin)[0].backward(ones[0])
    assert torch.equal(x.grad, abi.rdx_qk_norm_rope_grad(ones[0], 0 * ones[1], q, k, wq, wk, pos, cos, sin)[0])
    # no rotation, and on another stream
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    x = q.clone().requires_grad_()
    y, _ = abi.rdx_qk_norm_rope(x, k, wq, wk, None, None, None, stream=side)
    torch.cuda.current_stream(DEV).wait_stream(side)
    y.backward(ones[0])
    torch.cuda.synchronize()
    assert torch.equal(x.grad, abi.rdx_qk_norm_rope_grad(ones[0], 0 * ones[1], q, k, wq, wk, None, None, None)[0])
    with torch.no_grad():
        y, _ = abi.rdx_qk_norm_rope(x, k, wq, wk, pos, cos, sin, q_out=torch.empty_like(q))
    assert not y.requires_grad
    with pytest.raises(RuntimeError):
        abi.rdx_qk_norm_rope(x, k, wq, wk, pos, cos, sin, q_out=torch.empty_like(q))


def test_calls_that_write_into_tensors_tell_autograd():
    q, k, wq, wk, pos, cos, sin = qk_case(9, 4, 2, 64, 64, F32)
    _, cache, table, n = attend_case([9, 3], 4, 2, 64, 16, "int8", F32)

    def moves(call, *written):
        before = [x._version for x in written]
        call()
        assert all(x._version > b for x, b in zip(written, before))

    a, b, c, d = (torch.empty_like(x) for x in (q, k, wq, wk))
    moves(lambda: abi.rdx_qk_norm_rope(q, k, wq, wk, pos, cos, sin, q_out=a, k_out=b), a, b)
    moves(lambda: abi.rdx_qk_norm_rope_grad(q, k, q, k, wq, wk, pos, cos, sin, dq=a, dk=b, dq_weight=c, dk_weight=d), a, b, c, d)
    slots = torch.arange(9, device=DEV)
    moves(lambda: abi.rdx_kv_write(cache, k, k, slots), cache.k, cache.v, cache.k_scale, cache.v_scale)
    e = torch.empty_like(b)
    moves(lambda: abi.rdx_kv_read(cache, slots, dtype=F32, k_out=b, v_out=e), b, e)
    out, lse = torch.empty_like(q[:2]), torch.empty(2, 4, device=DEV)
    moves(lambda: abi.rdx_kv_attend(q[:2], cache, table, n, out=out, lse=lse), out, lse)
    # an operation that saved q for its gradient notices
    w = torch.ones_like(q).requires_grad_()
    loss = (q * w).sum()
    abi.rdx_qk_norm_rope(q, k, wq, wk, pos, cos, sin, q_out=q, k_out=k)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # tensors of inference mode have no counter
    with torch.inference_mode():
        a = torch.empty_like(q)
        abi.rdx_qk_norm_rope(q, k, wq, wk, pos, cos, sin, q_out=a, k_out=k)
    abi.rdx_qk_norm_rope(q, k, wq, wk, pos, cos, sin, q_out=a, k_out=k)


SLOW = """
#include <stdatomic.h>
#include <time.h>
static atomic_int entered, left;
int times_entered(void) { return entered; }
int times_left(void) { return left; }
int slow(const void* args, void* stream) {
    const struct timespec t = {0, 300000000};
    (void)args, (void)stream;
    atomic_fetch_add(&entered, 1);
    nanosleep(&t, 0);
    atomic_fetch_add(&left, 1);
    return 0;
}
"""


def test_other_threads_run_while_a_call_waits(tmp_path):
    # a launch waits where the queue before it is full; a stand-in for the library's entry waits 0.3 s
    (tmp_path / "slow.c").write_text(SLOW)
    subprocess.run([os.environ.get("CC", "gcc"), "-O1", "-shared", "-fPIC", str(tmp_path / "slow.c"), "-o",
                    str(tmp_path / "slow.so")], check=True)
    slow = ctypes.CDLL(str(tmp_path / "slow.so"))
    cache = abi.KVCache.zeros(1, 16, 2, 64, torch.int8, DEV)
    k, slots = torch.zeros(3, 2, 64, device=DEV), torch.arange(3, device=DEV)
    abi.rdx_kv_write(cache, k, k, slots)
    entries = [ctypes.cast(getattr(abi.load(), name), ctypes.c_void_p).value for name in abi.MARSHALLED]
    stand_in = ctypes.cast(slow.slow, ctypes.c_void_p).value
    module = abi._marshal()
    module.bind(*(stand_in if name == "rdx_kv_write" else e for name, e in zip(abi.MARSHALLED, entries)), abi.KVCache,
                abi._check)
    try:
        caller = threading.Thread(target=abi.rdx_kv_write, args=(cache, k, k, slots))
        caller.start()
        while slow.times_entered() == 0 and caller.is_alive():
            pass
        inside = slow.times_entered() == 1 and slow.times_left() == 0  # this thread runs, and the call is not back yet
        caller.join()
    finally:
        module.bind(*entries, abi.KVCache, abi._check)
    assert inside
    abi.rdx_kv_write(cache, k, k, slots)


def test_threads_and_streams_do_not_disturb_each_other():
    # four threads, each on a stream of its own with sizes of its own, through every operator; each result as alone
    def work(i, stream):
        q, k, wq, wk, pos, cos, sin = qk_case(50 + 300 * i, 8, 2, 64, 64, (F32, BF16)[i % 2], seed=i)
        x, cache, table, n = attend_case([200 + 900 * i, 31], 8, 2, 64, 16, "int8", (F32, BF16)[i % 2], seed=i)
        slots = torch.arange(q.shape[0], device=DEV)
        fresh = abi.KVCache.zeros(-(-q.shape[0] // 16), 16, 2, 64, torch.int8, DEV)
        torch.cuda.current_stream(DEV).synchronize()

        def once():
            a, b = abi.rdx_qk_norm_rope(q, k, wq, wk, pos, cos, sin, stream=stream)
            grads = abi.rdx_qk_norm_rope_grad(q, k, q, k, wq, wk, pos, cos, sin, stream=stream)
            abi.rdx_kv_write(fresh, k, b, slots, stream=stream)
            back = abi.rdx_kv_read(fresh, slots, dtype=F32, stream=stream)
            return (a, b, *grads, *back, abi.rdx_kv_attend(x, cache, table, n, stream=stream))

        return once

    streams = [torch.cuda.Stream(DEV) for _ in range(4)]
    calls = [work(i, s) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        for _ in range(20):
            got = calls[i]()
            streams[i].synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, alone[i])):
                wrong.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_rope_rows_past_the_range(dtype):
    # squares that pass float32's range: the row is zeros, as in plain float32 arithmetic; its neighbours are untouched
    q, k, wq, wk, pos, cos, sin = qk_case(5, 4, 2, 64, 64, dtype)
    want = abi.rdx_qk_norm_rope(q, k, wq, wk, pos, cos, sin)
    q[2, 1] = 2.0 ** 70
    got = abi.rdx_qk_norm_rope(q, k, wq, wk, pos, cos, sin)
    assert not got[0][2, 1].any()
    got[0][2, 1] = want[0][2, 1]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
