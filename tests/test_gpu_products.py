"""Grouped products of NVFP4 casts against fp64: nvfp4_group_gemm,
nvfp4_group_gated_gemm and nvfp4_group_wgrad, host-split and graph-safe."""
import pytest
import torch

from nvfp4_row_scaled_b200 import abi

from .products import COMPACT, TILED, check, product, random_matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_row_scaled_b200.build import build_library
    build_library()
    abi.lib()


def stacked(m, xv, wv, n):
    """fp64 product of the groups and its bound."""
    out, lim, o = [], [], 0
    for g, r in enumerate(m):
        p, b = product(xv[o:o + r], wv[g * n:(g + 1) * n])
        out.append(p)
        lim.append(b)
        o += r
    return torch.cat(out), torch.cat(lim)


def guarded(rows, cols, dtype, extra=3):
    """An output with `extra` rows behind it that must stay as they are."""
    t = torch.full((rows + extra, cols), 7.0, dtype=dtype, device="cuda")
    return t, t[:rows]


RAGGED = [
    ([1], 64, 16), ([1], 2048, 128), ([0, 1, 0], 256, 144), ([3, 17, 0, 300], 512, 272), ([255, 257], 320, 128),
    ([33], 4096, 1040), ([16, 16, 16], 96, 48), ([5, 0, 130], 48, 32), ([129], 16, 16), ([7, 9], 208, 112),
    ([1] * 40, 256, 160), ([600, 1], 1024, 256), ([0, 0], 64, 32), ([64], 7168, 64),
]


@pytest.mark.parametrize("m,K,N", RAGGED)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_any_group_sizes(m, K, N, dtype):
    rows, E = sum(m), len(m)
    x, xv = random_matrix(rows, K, 1 + K)
    w, wv = random_matrix(E * N, K, 2 + N)
    buf, y = guarded(rows, N, dtype)
    abi.nvfp4_group_gemm(x, m, w, y)
    want, lim = stacked(m, xv, wv, N)
    check(y, want, lim, f"{m} K={K} N={N}")
    assert bool((buf[rows:] == 7.0).all())


@pytest.mark.parametrize("xl,wl", [(TILED, TILED), (TILED, COMPACT), (COMPACT, TILED), (COMPACT, COMPACT)])
@pytest.mark.parametrize("m,K,N", [([128, 256, 0, 384], 512, 256), ([128], 128, 128), ([640, 128], 384, 384)])
def test_gemm_scale_layouts(m, K, N, xl, wl):
    rows, E = sum(m), len(m)
    x, xv = random_matrix(rows, K, 3, xl)
    w, wv = random_matrix(E * N, K, 4, wl)
    y = torch.full((rows, N), float("nan"), dtype=torch.float32, device="cuda")
    abi.nvfp4_group_gemm(x, m, w, y)
    check(y, *stacked(m, xv, wv, N), f"{xl} {wl}")


@pytest.mark.parametrize("m,K,F", [([1], 256, 16), ([3, 0, 70, 300], 512, 144), ([129, 5], 208, 48), ([1] * 20, 2048, 256)])
@pytest.mark.parametrize("save", [False, True])
def test_gated_any_group_sizes(m, K, F, save):
    run_gated(m, K, F, COMPACT, save)


@pytest.mark.parametrize("m,K,F", [([128, 0, 384], 256, 128), ([256], 1024, 384)])
def test_gated_tiled(m, K, F):
    run_gated(m, K, F, TILED, True)


def gated_reference(p, lim, F):
    """silu(g) u in fp64 with the bound carried through: |d silu| <= 1.1, and
    the kernel's fp32 exp, quotient and product add a few parts in 2^22 --
    the exponent's argument is rounded, |g| 2^-24, on top."""
    g, u = p[:, :F], p[:, F:]
    lg, lu = lim[:, :F], lim[:, F:]
    s = g * torch.sigmoid(g)
    h = s * u
    eps = (8 + g.abs()) * 2.0 ** -22
    return h, 1.1 * lg * (u.abs() + lu) + s.abs() * lu + eps * h.abs()


def run_gated(m, K, F, layout, save):
    rows, E = sum(m), len(m)
    x, xv = random_matrix(rows, K, 5, layout)
    w, wv = random_matrix(E * 2 * F, K, 6, layout)
    # pre-activations of ordinary size
    x["s2"] *= 2.0 ** -8
    xv = xv * 2.0 ** -8
    buf, h = guarded(rows, F, torch.bfloat16)
    pb, p = guarded(rows, 2 * F, torch.bfloat16)
    abi.nvfp4_group_gated_gemm(x, m, w, h, gate_up=p if save else None)
    want, lim = stacked(m, xv, wv, 2 * F)
    check(h, *gated_reference(want, lim, F), f"{m} K={K} F={F}")
    assert bool((buf[rows:] == 7.0).all())
    if save:
        check(p, want, lim, "gate_up")
        assert bool((pb[rows:] == 7.0).all())
    else:
        assert bool((pb == 7.0).all())


@pytest.mark.parametrize("m,N,K", [([16], 16, 16), ([16, 0, 48], 144, 272), ([128, 256], 128, 256), ([32, 80, 16], 48, 400),
                                   ([1040], 256, 128), ([0, 0], 32, 16), ([64, 128, 320], 304, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wgrad(m, N, K, dtype):
    run_wgrad(m, N, K, dtype, COMPACT, COMPACT)


@pytest.mark.parametrize("dl,xl", [(TILED, TILED), (TILED, COMPACT), (COMPACT, TILED)])
def test_wgrad_scale_layouts(dl, xl):
    run_wgrad([128, 0, 384], 256, 384, torch.float32, dl, xl)


def random_columns(m, width, seed, layout):
    """A column-wise cast: per group a [width, m_g] matrix."""
    parts = [random_matrix(width, r, seed + g, layout) for g, r in enumerate(m)]
    mats = [p[0] for p in parts]
    cat = {k: torch.cat([q[k].reshape(-1) for q in mats]) for k in ("data", "scale", "s2")}
    return abi.matrix(cat["data"], cat["scale"], cat["s2"], layout), [p[1] for p in parts]


def run_wgrad(m, N, K, dtype, dl, xl):
    E = len(m)
    dy, dv = random_columns(m, N, 100, dl)
    x, xv = random_columns(m, K, 200, xl)
    buf = torch.full((E * N * K + 64,), 7.0, dtype=dtype, device="cuda")
    dw = buf[:E * N * K].view(E, N, K)
    abi.nvfp4_group_wgrad(dy, x, m, dw)
    for g in range(E):
        want, lim = product(dv[g], xv[g])
        check(dw[g], want, lim, f"group {g}")
    assert bool((buf[E * N * K:] == 7.0).all())
