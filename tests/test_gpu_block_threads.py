"""The norms around a block called from two host threads at once, each on a stream of its own: the same kernel at two
widths, whose rings of shared memory differ in size. Each call gives what it gives alone. The C entry points are called
directly, so that the threads are in the library most of the time (a call there holds no lock of Python's)."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
CALLS = 20000
EPS = 1e-6


def join(moe, f, x, w, stream):
    lib, (T, H) = moe.load_library(), x.shape
    outs = [torch.empty_like(x), torch.empty_like(x)]
    p = moe.BlockJoinParams(w.data_ptr(), w.data_ptr(), None, 0, moe.MOE_F32, 1.0, 1.0, EPS)
    args = (f.data_ptr(), x.data_ptr(), moe.MOE_BF16, ctypes.byref(p), T, H, *(t.data_ptr() for t in outs),
            stream.cuda_stream)
    return lib.moe_block_join, args, outs, p


def join_backward(moe, f, x, w, stream):
    lib, (T, H) = moe.load_library(), x.shape
    ws = torch.empty(lib.moe_block_join_backward_workspace_size(T, H), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(x), torch.empty_like(x), torch.empty(H, device=DEV)]
    p = moe.BlockJoinParams(w.data_ptr(), None, None, 0, moe.MOE_F32, 1.0, 1.0, EPS)
    args = (x.data_ptr(), None, f.data_ptr(), None, moe.MOE_BF16, ctypes.byref(p), T, H, *(t.data_ptr() for t in outs),
            None, None, ws.data_ptr(), ws.numel(), stream.cuda_stream)
    return lib.moe_block_join_backward, args, outs, (p, ws)


@pytest.mark.parametrize("make,sizes", [(join, ((700, 4096), (3000, 1024))), (join_backward, ((700, 4096), (9000, 1024)))])
def test_two_threads_at_two_widths(cuda_lib, make, sizes):
    moe = cuda_lib
    jobs = []
    for seed, (T, H) in enumerate(sizes):
        rng = torch.Generator(DEV).manual_seed(seed)
        f, x = (torch.randn(T, H, generator=rng, device=DEV).bfloat16() for _ in range(2))
        w = torch.randn(H, generator=rng, device=DEV)
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        fn, args, outs, kept = make(moe, f, x, w, stream)
        assert fn(*args) == 0
        torch.cuda.synchronize()
        jobs.append((fn, args, outs, [t.clone() for t in outs], (f, x, w, stream, kept)))
    failed = [0, 0]
    start = threading.Barrier(2)

    def run(i):
        fn, args = jobs[i][:2]
        start.wait()
        failed[i] = sum(fn(*args) != 0 for _ in range(CALLS))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0]
    for _, _, outs, ref, _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    assert moe.moe_device_status() == 0
