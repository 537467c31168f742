"""Calls from several host threads at once: the library keeps nothing between calls,
and what the CUDA runtime keeps for a kernel (its limit of dynamic shared memory) does not
depend on the call."""
import os
import threading

import pytest
import torch

from nvfp4_row_scaled_b200 import abi

from .products import random_matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if os.environ.get("NVFP4RS_LIBRARY", "").endswith("_debug.so"):
        pytest.skip("the bounds-checked build keeps one table of ranges: one call at a time")
    from nvfp4_row_scaled_b200.build import build_library
    build_library()
    abi.lib()


def gemm(m, seed):
    x, _ = random_matrix(sum(m), 64, seed)
    w, _ = random_matrix(len(m) * 16, 64, seed + 1)
    y = torch.empty(sum(m), 16, device="cuda")
    return lambda s: abi.nvfp4_group_gemm(x, m, w, y, stream=s), [y]


def gated(m, seed):
    x, _ = random_matrix(sum(m), 64, seed)
    w, _ = random_matrix(len(m) * 32, 64, seed + 1)
    h = torch.empty(sum(m), 16, dtype=torch.bfloat16, device="cuda")
    return lambda s: abi.nvfp4_group_gated_gemm(x, m, w, h, stream=s), [h]


def backward(m, F, seed):
    g = torch.Generator().manual_seed(seed)
    dh, gu = (torch.randn(sum(m), n, generator=g).to(torch.bfloat16).cuda() for n in (F, 2 * F))
    d, (ra, ca) = torch.empty_like(gu), abi.alloc_amax(sum(m), 2 * F, len(m))
    return lambda s: abi.nvfp4_group_gated_backward(dh, gu, m, d, ra, ca, stream=s), [d, ra, ca]


def cast(m, K, seed, mx=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(sum(m), K, generator=g).to(torch.bfloat16).cuda()
    if mx:
        out = abi.alloc_mx_outputs(sum(m), K)
        return lambda s: abi.nvfp4_mx_group_cast(x, m, out, stream=s), list(out.values())
    (ra, ca), out = abi.alloc_amax(sum(m), K, len(m)), abi.alloc_outputs(sum(m), K, len(m))

    def call(s):
        abi.nvfp4_group_amax(x, m, ra, ca, stream=s)
        abi.nvfp4_group_cast(x, m, ra, ca, out, stream=s)
    return call, [ra, ca, *out.values()]


def quantize(m, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(sum(m), K, generator=g).to(torch.bfloat16).cuda()
    (ra, ca), out, ws = abi.alloc_amax(sum(m), K, len(m)), abi.alloc_outputs(sum(m), K, len(m)), abi.alloc_workspace(0, len(m))
    return lambda s: abi.nvfp4_group_quantize(x, m, ra, ca, out, ws, stream=s), [ra, ca, *out.values()]


few, many = [16], [16] + [0] * 1022 + [16]
CALLS = {
    "gemm": lambda: [gemm(few, 1), gemm(many, 2)],
    "gated": lambda: [gated(few, 3), gated(many, 4)],
    "gated_backward": lambda: [backward([16], 48 * 1024, 5), backward([16], 65536, 6)],
    "cast": lambda: [cast(few, 64, 7), cast(many, 64, 8)],
    "amax_of_wide_rows": lambda: [cast(few, 128 * 113, 9), cast(few, 128 * 227, 10)],
    "mx_cast": lambda: [cast([32], 64, 11, True), cast([32] + [0] * 1023, 64, 12, True)],
    "quantize": lambda: [quantize([128], 128, 13), quantize([128] + [0] * 1023, 128, 14)],
}


@pytest.mark.parametrize("what", sorted(CALLS))
def test_two_threads_with_calls_of_different_sizes(what):
    """Two host threads, a stream each, the kernel's smallest and largest launches side
    by side: none fails, and the outputs are those of one call after the other."""
    calls = CALLS[what]()
    want = []
    for call, outs in calls:
        call(None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.view(torch.uint8).fill_(0xA5)
    errors, start = [], threading.Barrier(len(calls))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def loop(call, stream):
        try:
            stream.synchronize()
            start.wait()
            for _ in range(1500):
                call(stream)
        except Exception as e:  # noqa: BLE001 - reported by the test's thread
            errors.append(e)
    threads = [threading.Thread(target=loop, args=(c[0], s)) for c, s in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    for (_, outs), w in zip(calls, want):
        for a, b in zip(outs, w):
            assert torch.equal(a, b)


def cast_only(m, K, seed):
    call, outs = cast(m, K, seed)
    call(None)
    x = torch.randn(sum(m), K, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    ra, ca = outs[:2]
    out = abi.alloc_outputs(sum(m), K, len(m))
    return lambda s: abi.nvfp4_group_cast(x, m, ra, ca, out, stream=s), list(out.values())


def wgrad(m, seed):
    q = [random_matrix(32, sum(m), seed + i)[0] for i in range(2)]
    dw = torch.empty(1, 32, 32, device="cuda")
    return lambda s: abi.nvfp4_group_wgrad(*q, m, dw, stream=s), [dw]


def gemm_odd(seed):
    x, _ = random_matrix(5, 48, seed)
    w, _ = random_matrix(16, 48, seed + 1)
    y = torch.empty(5, 16, device="cuda")
    return lambda s: abi.nvfp4_group_gemm(x, [5], w, y, stream=s), [y]


FIRST = {
    "gemm": lambda: gemm([7], 1), "gemm_without_maps": lambda: gemm_odd(2), "gated": lambda: gated([7], 3),
    "wgrad": lambda: wgrad([64], 4), "gated_backward": lambda: backward([16], 64, 5), "cast": lambda: cast([16], 64, 6),
    "cast_alone": lambda: cast_only([16], 64, 7), "mx_cast": lambda: cast([32], 64, 8, True), "quantize": lambda: quantize([128], 128, 9),
}


@pytest.mark.parametrize("what", sorted(FIRST))
def test_first_cuda_call_of_a_thread(what):
    """A call from a host thread that has made no CUDA call before."""
    call, outs = FIRST[what]()
    call(None)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.view(torch.uint8).fill_(0xA5)
    torch.cuda.synchronize()
    stream, errors = torch.cuda.Stream(), []

    def first():
        try:
            call(stream)
        except Exception as e:  # noqa: BLE001 - reported by the test's thread
            errors.append(e)
    t = threading.Thread(target=first)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
