"""Refusals of the products, found on the host before anything is enqueued (no
call here reaches the CUDA runtime), and the binding's checks."""
import ctypes

import pytest
import torch

from nvfp4_row_scaled_b200 import abi
from nvfp4_row_scaled_b200.build import build_library

OK, BAD, UNS = abi.NVFP4_OK, abi.NVFP4_ERR_INVALID_ARG, abi.NVFP4_ERR_UNSUPPORTED
FAKE = 0x10000  # 16-byte aligned, never dereferenced
TILED = abi.NVFP4_SCALE_TILED_128X4
F32, BF16 = abi.NVFP4_OUT_F32, abi.NVFP4_OUT_BF16


@pytest.fixture(scope="module")
def L():
    build_library()
    return abi.lib()


def mat(layout=0, data=FAKE, scale=FAKE, s2=FAKE):
    return abi.Matrix(data, scale, s2, layout)


def splits(m):
    return (ctypes.c_int64 * max(len(m), 1))(*m)


GEMM = [
    (dict(K=24), BAD), (dict(N=24), BAD), (dict(rows=-1), BAD), (dict(m=[40, 40]), BAD), (dict(m=[-1, 65]), BAD),
    (dict(K=-16), BAD), (dict(N=-16), BAD), (dict(y=None), BAD), (dict(dtype=2), BAD), (dict(x=None), BAD),
    (dict(x=mat(data=None)), BAD), (dict(w=mat(scale=None)), BAD), (dict(w=mat(s2=None)), BAD), (dict(x=mat(layout=2)), BAD),
    (dict(x=mat(data=FAKE + 8)), UNS), (dict(w=mat(scale=FAKE + 4)), UNS), (dict(x=mat(s2=FAKE + 2)), UNS),
    (dict(y=FAKE + 8), UNS), (dict(x=mat(TILED), m=[64]), UNS), (dict(x=mat(TILED), m=[128], rows=128, K=64), UNS),
    (dict(w=mat(TILED), N=64, K=128), UNS), (dict(m=[0] * 1025 + [64]), UNS), (dict(N=1 << 30, m=[64, 0, 0]), UNS),
    (dict(rows=(1 << 31) - 1000, m=[(1 << 31) - 1000]), UNS),
    (dict(rows=0, m=[0, 0]), OK), (dict(N=0), OK), (dict(rows=0, m=[]), OK),
]


@pytest.mark.parametrize("change,want", GEMM)
def test_gemm_host_checks(L, change, want):
    c = dict(x=mat(), rows=64, K=128, m=[64], w=mat(), N=32, y=FAKE, dtype=BF16)
    c.update(change)
    assert L.nvfp4_group_gemm(c["x"], c["rows"], c["K"], splits(c["m"]), len(c["m"]), c["w"], c["N"], c["y"], c["dtype"],
                              None) == want


@pytest.mark.parametrize("change,want", [
    (dict(K=0), BAD), (dict(status=None), BAD), (dict(fd=None), BAD), (dict(to=None), BAD), (dict(to=FAKE + 4), UNS),
    (dict(fd=None, to=None, E=3), BAD), (dict(fd=None, to=None, E=2, x=mat(TILED)), UNS), (dict(E=1025), UNS), (dict(E=-1), BAD),
])
def test_gemm_graphsafe_host_checks(L, change, want):
    c = dict(x=mat(), rows=64, K=128, fd=FAKE, to=FAKE, E=2, w=mat(), N=32, y=FAKE, status=FAKE)
    c.update(change)
    for out in (c["y"],):
        assert L.nvfp4_group_gemm_graphsafe(c["x"], c["rows"], c["K"], c["fd"], c["to"], c["E"], c["w"], c["N"], out, BF16,
                                            c["status"], None) == want
        assert L.nvfp4_group_gated_gemm_graphsafe(c["x"], c["rows"], c["K"], c["fd"], c["to"], c["E"], c["w"], c["N"], out,
                                                  None, c["status"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(F=24), BAD), (dict(F=-16), BAD), (dict(h=None), BAD), (dict(K=40), BAD), (dict(gate_up=FAKE + 8), UNS),
    (dict(w=mat(TILED), F=64), UNS), (dict(m=[63]), BAD), (dict(rows=0, m=[0]), OK), (dict(F=0), OK),
])
def test_gated_host_checks(L, change, want):
    c = dict(rows=64, K=128, m=[64], w=mat(), F=32, h=FAKE, gate_up=FAKE)
    c.update(change)
    assert L.nvfp4_group_gated_gemm(mat(), c["rows"], c["K"], splits(c["m"]), len(c["m"]), c["w"], c["F"], c["h"],
                                    c["gate_up"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(N=24), BAD), (dict(K=24), BAD), (dict(m=[40]), BAD), (dict(m=[40, 24]), UNS), (dict(dw=None), BAD),
    (dict(dw=None, rows=0, m=[0]), BAD), (dict(dtype=7), BAD), (dict(dy=mat(data=None)), BAD), (dict(x=mat(s2=None)), BAD),
    (dict(x=mat(TILED), rows=128, m=[128], K=64), UNS), (dict(dy=mat(TILED), N=128, K=128), UNS), (dict(m=[-16, 80]), BAD),
    (dict(E0=True, m=[], rows=0), OK), (dict(N=0), OK), (dict(K=0), OK),
])
def test_wgrad_host_checks(L, change, want):
    c = dict(dy=mat(), x=mat(), rows=64, m=[64], N=32, K=48, dw=FAKE, dtype=F32)
    c.update(change)
    assert L.nvfp4_group_wgrad(c["dy"], c["x"], c["rows"], splits(c["m"]), len(c["m"]), c["N"], c["K"], c["dw"], c["dtype"],
                               None) == want


@pytest.mark.parametrize("change,want", [
    (dict(F=24), BAD), (dict(F=-16), BAD), (dict(dh=None), BAD), (dict(gu=None), BAD), (dict(d=None), BAD), (dict(m=[24, 40]), UNS),
    (dict(m=[48]), BAD), (dict(F=65552), UNS), (dict(dh=FAKE + 8), UNS), (dict(ra=FAKE + 2), UNS), (dict(F=0), OK),
])
def test_gated_backward_host_checks(L, change, want):
    c = dict(dh=FAKE, gu=FAKE, rows=64, F=32, m=[64], d=FAKE, ra=FAKE, ca=FAKE)
    c.update(change)
    assert L.nvfp4_group_gated_backward(c["dh"], c["gu"], c["rows"], c["F"], splits(c["m"]), len(c["m"]), c["d"], c["ra"],
                                        c["ca"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(rank=12), BAD), (dict(rank=0), BAD), (dict(rank=72), UNS), (dict(ids=None), BAD), (dict(ws=None), BAD),
    (dict(wsb=64 * 16 * 4 - 1), BAD), (dict(status=None), BAD), (dict(a=None), BAD), (dict(b=None), BAD), (dict(f=None), BAD),
    (dict(xb=None), BAD), (dict(L=-1), BAD), (dict(K=24), BAD), (dict(N=8), BAD), (dict(y=None), BAD), (dict(dtype=3), BAD),
    (dict(a=FAKE + 8), UNS), (dict(b=FAKE + 2), UNS), (dict(ws=FAKE + 4), UNS), (dict(x=mat(TILED), K=128), UNS),
])
def test_adapter_host_checks(L, change, want):
    c = dict(xb=FAKE, x=mat(), rows=64, K=32, N=16, a=FAKE, b=FAKE, f=FAKE, L=2, rank=16, ids=FAKE, y=FAKE, dtype=BF16, ws=FAKE,
             wsb=64 * 16 * 4, status=FAKE)
    c.update(change)
    assert L.nvfp4_adapter_gemm(c["xb"], c["x"], c["rows"], c["K"], mat(), c["N"], c["a"], c["b"], c["f"], c["L"], c["rank"],
                                c["ids"], c["y"], c["dtype"], c["ws"], c["wsb"], c["status"], None) == want


def test_adapter_workspace_bytes(L):
    assert abi.nvfp4_adapter_workspace_bytes(7, 16) == 7 * 16 * 4
    assert abi.nvfp4_adapter_workspace_bytes(0, 16) == 0
    for rows, rank in ((-1, 16), (4, -8), (4, 72), (1 << 31, 8)):
        assert abi.nvfp4_adapter_workspace_bytes(rows, rank) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes(L):
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)  # noqa: E731
    x = abi.matrix(z(4, 32), z(4, 4), z(4, dt=torch.float32))
    w = abi.matrix(z(16, 32), z(16, 4), z(16, dt=torch.float32))
    y = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        abi.nvfp4_group_gemm(x, [4], w, y)
    with pytest.raises(ValueError, match="CUDA"):
        abi.nvfp4_group_gated_backward(torch.zeros(16, 16), torch.zeros(16, 32), [16], torch.zeros(16, 32))
    cuda0 = torch.device("cuda:0")
    with pytest.raises(ValueError, match="must hold"):
        abi._matrix(x, 5, 5 * 64, cuda0, "x")
    with pytest.raises(ValueError, match="must be on"):
        abi._matrix(x, 4, 4 * 64, cuda0, "x")
    with pytest.raises(ValueError, match="equal rows"):
        abi._width(w, x, 3)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        abi._out_dtype(torch.zeros(1, dtype=torch.float16), "y")


@pytest.mark.parametrize("m", [[64, (1 << 63) - 1, (1 << 63) - 1, 2], [64, (1 << 63) - 16, (1 << 63) - 16, 32], [16, (1 << 63) - 16, 64]])
def test_splits_whose_sum_overflows(L, m):
    """Sizes that add up to 64 only modulo 2^64 are refused by every host-split call."""
    out = abi.Outputs(row_data=FAKE, row_scale=FAKE, row_s2=FAKE)
    mx = abi.MxOutputs(row_data=FAKE, row_scale=FAKE)
    n, ap = len(m), splits(m)
    assert L.nvfp4_group_gemm(mat(), 64, 128, ap, n, mat(), 32, FAKE, BF16, None) == BAD
    assert L.nvfp4_group_gated_gemm(mat(), 64, 128, ap, n, mat(), 32, FAKE, FAKE, None) == BAD
    assert L.nvfp4_group_wgrad(mat(), mat(), 64, ap, n, 32, 48, FAKE, F32, None) == BAD
    assert L.nvfp4_group_gated_backward(FAKE, FAKE, 64, 32, ap, n, FAKE, FAKE, FAKE, None) == BAD
    assert L.nvfp4_group_amax(FAKE, 64, 128, ap, n, FAKE, FAKE, None) == BAD
    assert L.nvfp4_group_cast(FAKE, 64, 128, ap, n, FAKE, FAKE, ctypes.byref(out), None) == BAD
    assert L.nvfp4_mx_group_cast(FAKE, 64, 128, ap, n, ctypes.byref(mx), None) == BAD


def test_calls_run_on_the_tensors_device(monkeypatch):
    """Tensors on a device that is not the current one: the call is made with that device current, on its
    current stream, and the former device is current again; a stream of another device is refused."""
    state, seen = {"current": 0}, []

    class Guard:
        def __init__(self, dev):
            self.dev = torch.device(dev).index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.dev

        def __exit__(self, *exc):
            state["current"] = self.before
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)

    def entry(*args):
        seen.append((state["current"], args))
        return OK
    one = torch.device("cuda:1")
    abi._run(one, None, "call", entry, 7)
    assert seen == [(1, (7, 1001))] and state["current"] == 0

    class Stream:
        cuda_stream = 55

        def __init__(self, index):
            self.device = torch.device("cuda", index)
    abi._run(one, Stream(1), "call", entry)
    assert seen[-1] == (1, (55,)) and state["current"] == 0
    with pytest.raises(ValueError, match="stream is on"):
        abi._run(one, Stream(0), "call", entry)

    def fails(*args):
        return abi.NVFP4_ERR_UNSUPPORTED
    with pytest.raises(abi.NVFP4Error):
        abi._run(one, None, "call", fails)
    assert state["current"] == 0 and len(seen) == 2
