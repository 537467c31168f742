"""Grouped products of NVFP4 casts against fp64: nvfp4_group_gemm,
nvfp4_group_gated_gemm and nvfp4_group_wgrad, host-split and graph-safe."""
import os

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


# ----------------------------------------------------------------- routing

def routings(m, K, rows):
    fd, offs = abi.routing_tensors(m, K)
    return fd, offs, torch.full((1,), -1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("m,cap", [([3, 0, 70, 300], 400), ([0, 0, 0], 64), ([128, 128], 256)])
def test_graphsafe_equals_host_split(m, cap):
    """The same bits for the same routing; rows behind the routed total stay."""
    K, N, E, rows = 512, 144, len(m), sum(m)
    x, _ = random_matrix(cap, K, 7)
    w, _ = random_matrix(E * 2 * N, K, 8)
    w1 = abi.matrix(w["data"][:E * N].contiguous(), w["scale"][:E * N].contiguous(), w["s2"][:E * N].contiguous())
    xr = abi.matrix(x["data"][:rows].contiguous(), x["scale"][:rows].contiguous(), x["s2"][:rows].contiguous())
    fd, offs, st = routings(m, K, rows)
    y = torch.full((cap, N), 7.0, device="cuda")
    yh = torch.empty(rows, N, device="cuda")
    abi.nvfp4_group_gemm_graphsafe(x, fd, offs, w1, y, st)
    abi.nvfp4_group_gemm(xr, m, w1, yh)
    assert int(st.item()) == 0
    assert torch.equal(y[:rows], yh) and bool((y[rows:] == 7.0).all())
    h = torch.full((cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
    p = torch.full((cap, 2 * N), 7.0, dtype=torch.bfloat16, device="cuda")
    hh, ph = h[:rows].clone(), p[:rows].clone()
    abi.nvfp4_group_gated_gemm_graphsafe(x, fd, offs, w, h, st, gate_up=p)
    abi.nvfp4_group_gated_gemm(xr, m, w, hh, gate_up=ph)
    assert int(st.item()) == 0
    assert torch.equal(h[:rows], hh) and torch.equal(p[:rows], ph)
    assert bool((h[rows:] == 7.0).all()) and bool((p[rows:] == 7.0).all())


@pytest.mark.parametrize("fault", ["offset", "first", "beyond"])
def test_graphsafe_bad_routing_writes_nothing(fault):
    K, N = 128, 32
    x, _ = random_matrix(64, K, 9)
    w, _ = random_matrix(2 * 2 * N, K, 10)
    w1 = abi.matrix(w["data"][:2 * N].contiguous(), w["scale"][:2 * N].contiguous(), w["s2"][:2 * N].contiguous())
    fd, offs, st = routings([32, 32], K, 64)
    if fault == "offset":
        offs[1] += 1
    elif fault == "first":
        fd[0] = 16
    else:
        fd[1], offs[2] = 48, 80 * K
    y = torch.full((64, N), 7.0, device="cuda")
    abi.nvfp4_group_gemm_graphsafe(x, fd, offs, w1, y, st)
    assert int(st.item()) == abi.NVFP4_ERR_ROUTING and bool((y == 7.0).all())
    h = torch.full((64, N), 7.0, dtype=torch.bfloat16, device="cuda")
    abi.nvfp4_group_gated_gemm_graphsafe(x, fd, offs, w, h, st)
    assert int(st.item()) == abi.NVFP4_ERR_ROUTING and bool((h == 7.0).all())


def test_graphsafe_tiled_rows_need_128():
    x, _ = random_matrix(256, 128, 11, TILED)
    w, _ = random_matrix(2 * 128, 128, 12, TILED)
    fd, offs, st = routings([64, 192], 128, 256)
    y = torch.full((256, 128), 7.0, device="cuda")
    abi.nvfp4_group_gemm_graphsafe(x, fd, offs, w, y, st)
    assert int(st.item()) == abi.NVFP4_ERR_UNSUPPORTED and bool((y == 7.0).all())


def test_uniform_groups():
    x, xv = random_matrix(96, 64, 13)
    w, wv = random_matrix(3 * 48, 64, 14)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.empty(96, 48, device="cuda")
    abi.nvfp4_group_gemm_graphsafe(x, None, None, w, y, st, num_groups=3)
    assert int(st.item()) == 0
    check(y, *stacked([32] * 3, xv, wv, 48))


def test_wgrad_graphsafe_equals_host_split():
    m, N, K = [48, 0, 160], 144, 80
    dy, _ = random_columns(m, N, 300, COMPACT)
    x, _ = random_columns(m, K, 400, COMPACT)
    fd, offs, st = routings(m, K, sum(m))
    a, b = torch.full((3, N, K), 7.0, device="cuda"), torch.empty(3, N, K, device="cuda")
    abi.nvfp4_group_wgrad_graphsafe(dy, x, sum(m), fd, offs, a, st)
    abi.nvfp4_group_wgrad(dy, x, m, b)
    assert int(st.item()) == 0 and torch.equal(a, b) and bool((a[1] == 0).all())
    fd[0], offs[1] = 40, 40 * K  # not a multiple of 16 rows
    a.fill_(7.0)
    fd[2], offs[3] = 168, 208 * K
    abi.nvfp4_group_wgrad_graphsafe(dy, x, sum(m), fd, offs, a, st)
    assert int(st.item()) != 0
    fd[2] = 168
    offs[2] = 40 * K
    abi.nvfp4_group_wgrad_graphsafe(dy, x, sum(m), fd, offs, a, st)
    assert int(st.item()) in (abi.NVFP4_ERR_UNSUPPORTED, abi.NVFP4_ERR_ROUTING) and bool((a == 7.0).all())


def test_graph_replays_with_other_routings():
    """One captured graph, the routing rewritten between replays."""
    K, N, E, cap = 256, 64, 4, 200
    x, xv = random_matrix(cap, K, 15)
    w, wv = random_matrix(E * N, K, 16)
    fd, offs, st = routings([50] * 4, K, cap)
    y = torch.empty(cap, N, device="cuda")
    abi.nvfp4_group_gemm_graphsafe(x, fd, offs, w, y, st)  # before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.nvfp4_group_gemm_graphsafe(x, fd, offs, w, y, st)
    for m in ([200, 0, 0, 0], [1, 2, 3, 4], [0, 99, 0, 101], [0, 0, 0, 0]):
        f2, o2 = abi.routing_tensors(m, K)
        fd.copy_(f2)
        offs.copy_(o2)
        y.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        n = sum(m)
        if n:
            check(y[:n], *stacked(m, xv, wv, N), str(m))
        assert bool((y[n:] == 7.0).all())


def test_zero_contraction_gives_zeros():
    x, _ = random_matrix(5, 0, 17)
    w, _ = random_matrix(2 * 32, 0, 18)
    y = torch.full((5, 32), 7.0, device="cuda")
    abi.nvfp4_group_gemm(x, [5, 0], w, y)
    assert bool((y == 0).all())


def test_nan_scale_stays_in_its_rows():
    """A NaN block scale of one token or one weight row reaches that row and column only."""
    x, xv = random_matrix(300, 256, 19)
    w, wv = random_matrix(160, 256, 20)
    x["scale"][17, 3] = 0x7F
    w["scale"][130, 1] = 0x7F
    y = torch.empty(300, 160, device="cuda")
    abi.nvfp4_group_gemm(x, [300], w, y)
    nan = torch.isnan(y.cpu())
    want = torch.zeros(300, 160, dtype=torch.bool)
    want[17], want[:, 130] = True, True
    assert torch.equal(nan, want)
    p, b = product(xv, wv)
    keep = ~want
    check(y.cpu()[keep], p[keep], b[keep])


def test_two_streams_at_once():
    """Calls on two streams share nothing."""
    if os.environ.get("NVFP4RS_LIBRARY"):
        pytest.skip("the bounds-checked build keeps one table of ranges: one call at a time")
    K, N = 1024, 256
    ins = [(random_matrix(200, K, 21 + i), random_matrix(N, K, 31 + i)) for i in range(2)]
    ys = [torch.empty(200, N, device="cuda") for _ in range(2)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            abi.nvfp4_group_gemm(ins[i][0][0], [200], ins[i][1][0], ys[i], stream=ss[i])
    torch.cuda.synchronize()
    for i in range(2):
        check(ys[i], *product(ins[i][0][1], ins[i][1][1]), f"stream {i}")


def test_offsets_past_32_bits():
    """The last rows of an output of more than 2^31 elements, and of weights of
    more than 2^32 codes."""
    K, N, rows = 32, 16400, 131200
    x, xv = random_matrix(64, K, 22)
    big = abi.matrix(*(torch.cat([torch.zeros(rows - 64, *x[k].shape[1:], dtype=x[k].dtype, device="cuda"), x[k]])
                       for k in ("data", "scale", "s2")))
    w, wv = random_matrix(N, K, 23)
    y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    abi.nvfp4_group_gemm(big, [rows], w, y)
    check(y[-64:], *product(xv, wv))
    assert bool((y[:64] == 0).all())
    del y, big
    E, N, K = 70, 16384, 4096
    wl, wlv = random_matrix(N, K, 24)
    rep = abi.matrix(*(torch.cat([torch.zeros((E - 1) * N, *wl[k].shape[1:], dtype=wl[k].dtype, device="cuda"), wl[k]])
                       for k in ("data", "scale", "s2")))
    x, xv = random_matrix(5, K, 25)
    y = torch.empty(5, N, device="cuda")
    abi.nvfp4_group_gemm(x, [0] * (E - 1) + [5], rep, y)
    check(y, *product(xv, wlv))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_do_not_depend_on_the_size_of_the_call(dtype):
    """The same bits from a call large enough for pairs of CTAs, from a few rows and
    from one."""
    K, N, rows = 1056, 2064, 4100
    x, xv = random_matrix(rows, K, 26)
    w, wv = random_matrix(N, K, 27)
    y = torch.empty(rows, N, dtype=dtype, device="cuda")
    abi.nvfp4_group_gemm(x, [rows], w, y)
    check(y[-300:], *product(xv[-300:], wv), "large")
    for lo, hi in ((0, 1), (7, 60), (4000, 4100)):
        part = abi.matrix(*(x[k][lo:hi].clone() for k in ("data", "scale", "s2")))  # 16-byte aligned copies
        z = torch.empty(hi - lo, N, dtype=dtype, device="cuda")
        abi.nvfp4_group_gemm(part, [hi - lo], w, z)
        assert torch.equal(z, y[lo:hi]), (lo, hi)


def test_large_gated_and_wgrad_pairs():
    """Pairs of CTAs with ragged ends on both sides, empty groups among them."""
    m, K, F = [700, 0, 1, 900, 333], 544, 1040
    run_gated(m, K, F, COMPACT, True)
    run_wgrad([304, 0, 512, 16], 1552, 1296, torch.bfloat16, COMPACT, COMPACT)
    run_wgrad([256, 0, 512], 1536, 1280, torch.float32, TILED, TILED)


def test_gated_at_every_gate():
    """Gates from -1400 to 1400, those among them at which e^-g is above 2^126 or
    infinite and e^g below 2^-126, with up projections large enough that the product is an ordinary number:
    h is held to the bound of gated_reference and half a step, with no absolute allowance."""
    K, F, rows = 16, 64, 48
    x, _ = random_matrix(rows, K, 28)
    w, _ = random_matrix(2 * F, K, 29)
    x["data"].fill_(0x22)  # 1.0
    x["scale"].fill_(0x38)  # 1.0
    x["s2"].fill_(2.0 ** -4)
    w["data"].fill_(0x22)
    w["scale"].fill_(0x38)
    gate = torch.cat([torch.tensor([-1400.0, -300.0, -170.0, -104.0, -103.0, -90.0, -88.5, -88.0, -87.5, -87.0, -86.0, -30.0, -1.0,
                                    -0.0, 1e-30, 0.5, 20.0, 87.0, 87.5, 88.5, 89.0, 104.0, 1400.0]),
                      torch.linspace(-120, 120, F - 23)])
    up = torch.cat([torch.full((12,), 2.0 ** 120), torch.ones(11), torch.full((F - 23,), 2.0 ** 60)])
    w["s2"][:F], w["s2"][F:] = gate.cuda(), up.cuda()
    h = torch.empty(rows, F, dtype=torch.bfloat16, device="cuda")
    abi.nvfp4_group_gated_gemm(x, [rows], w, h)
    p = torch.cat([gate, up]).double().expand(rows, -1)  # 16 ones, times 2^-4, times the factor: exact
    want, lim = gated_reference(p, torch.zeros(rows, 2 * F, dtype=torch.float64), F)
    got = h.double().cpu()
    # the smallest normal bf16 is 2^-126; below it steps of 2^-133
    err, room = (got - want).abs(), lim + 2.0 ** -8 * (want.abs() + lim) + 2.0 ** -134
    assert bool((err <= room).all()), (gate[(err > room)[0]], got[0][(err > room)[0]], want[0][(err > room)[0]])


@pytest.mark.parametrize("m,K", [([1], 16), ([3], 48), ([129], 16), ([5, 0, 6], 80), ([2], 1040), ([131], 176), ([7], 1008),
                                 ([66, 1], 272), ([257], 304)])
def test_scales_that_end_inside_a_word(m, K):
    """Row-major scales whose matrix ends 1, 2 or 3 bytes into an aligned word, NaN bytes behind
    them: the values are right, and the bounds-checked build counts a read behind them."""
    rows, E, N = sum(m), len(m), 48
    assert rows * (K // 16) % 4
    x, xv = random_matrix(rows, K, 30)
    w, wv = random_matrix(E * 2 * N, K, 31)
    n = x["scale"].numel()
    buf = torch.full((n + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    buf[:n] = x["scale"].view(-1)
    x["scale"] = buf[:n].view(rows, K // 16)
    want, lim = stacked(m, xv, wv, 2 * N)
    y = torch.empty(rows, 2 * N, device="cuda")
    abi.nvfp4_group_gemm(x, m, w, y)
    check(y, want, lim)
    fd, offs, st = routings(m, K, rows)
    z = torch.empty_like(y)
    abi.nvfp4_group_gemm_graphsafe(x, fd, offs, w, z, st)
    assert int(st.item()) == 0 and torch.equal(y, z)
    x["s2"] *= 2.0 ** -8
    h, p = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, 2 * N, dtype=torch.bfloat16, device="cuda")
    abi.nvfp4_group_gated_gemm(x, m, w, h, gate_up=p)
    want, lim = stacked(m, xv * 2.0 ** -8, wv, 2 * N)
    check(p, want, lim)
    check(h, *gated_reference(want, lim, N))


def test_graphsafe_without_groups_writes_nothing():
    """No groups, rows allocated: nothing is routed, so nothing is written, as in the casts."""
    K, N, cap = 64, 32, 40
    x, _ = random_matrix(cap, K, 32)
    w, _ = random_matrix(0, K, 33)
    fd, offs = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    for arrays in ((fd, offs), (None, None)):
        st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        y = torch.full((cap, N), 7.0, device="cuda")
        abi.nvfp4_group_gemm_graphsafe(x, *arrays, w, y, st, num_groups=0)
        h = torch.full((cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
        abi.nvfp4_group_gated_gemm_graphsafe(x, *arrays, w, h, st, num_groups=0)
        assert int(st.item()) == 0 and bool((y == 7.0).all()) and bool((h == 7.0).all())


def test_longest_contraction():
    """The longest K: a tile's products take a second, and the warps that wait for them wait that
    long. Ones at both ends, zeros between."""
    K, N = 1 << 30, 16
    x = abi.matrix(torch.zeros(1, K // 2, dtype=torch.uint8, device="cuda"), torch.full((1, K // 16), 0x38, dtype=torch.uint8, device="cuda"),
                   torch.ones(1, device="cuda"))
    w = abi.matrix(torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"), torch.full((N, K // 16), 0x38, dtype=torch.uint8, device="cuda"),
                   torch.arange(1.0, N + 1, device="cuda"))
    for t in (x["data"], w["data"]):
        t[:, :100] = 0x22
        t[:, -60:] = 0x22
    y = torch.full((1, N), 7.0, device="cuda")
    abi.nvfp4_group_gemm(x, [1], w, y)
    assert torch.equal(y.cpu(), 320.0 * torch.arange(1.0, N + 1)[None])


def test_1024_groups():
    """As many groups as a call takes, most of them empty or of one row, host-split and graph-safe."""
    E, K, N = 1024, 64, 32
    m = [(0, 1, 0, 3)[g % 4] for g in range(E)]
    m[500], m[-1] = 140, 33
    rows = sum(m)
    x, xv = random_matrix(rows, K, 34)
    w, wv = random_matrix(E * N, K, 35)
    buf, y = guarded(rows, N, torch.float32)
    abi.nvfp4_group_gemm(x, m, w, y)
    check(y, *stacked(m, xv, wv, N))
    assert bool((buf[rows:] == 7.0).all())
    fd, offs, st = routings(m, K, rows)
    z = torch.empty_like(y)
    abi.nvfp4_group_gemm_graphsafe(x, fd, offs, w, z, st)
    assert int(st.item()) == 0 and torch.equal(y, z)
    run_wgrad([0, 16, 0, 0] * 255 + [48, 0, 16, 0], 32, 16, torch.float32, COMPACT, COMPACT)


def test_gated_rows_do_not_depend_on_the_size_of_the_call():
    """The same bits from a call large enough for pairs of CTAs, from a few rows and from one."""
    K, F, rows = 1056, 1040, 4100
    x, _ = random_matrix(rows, K, 36)
    x["s2"] *= 2.0 ** -8
    w, _ = random_matrix(2 * F, K, 37)
    h, p = torch.empty(rows, F, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, 2 * F, dtype=torch.bfloat16, device="cuda")
    abi.nvfp4_group_gated_gemm(x, [rows], w, h, gate_up=p)
    for lo, hi in ((0, 1), (7, 60), (4000, 4100)):
        part = abi.matrix(*(x[k][lo:hi].clone() for k in ("data", "scale", "s2")))
        h2, p2 = torch.empty_like(h[lo:hi]), torch.empty_like(p[lo:hi])
        abi.nvfp4_group_gated_gemm(part, [hi - lo], w, h2, gate_up=p2)
        assert torch.equal(h2, h[lo:hi]) and torch.equal(p2, p[lo:hi]), (lo, hi)


def test_weight_gradient_does_not_depend_on_the_other_groups():
    """A group's gradient among 40 groups (pairs of CTAs) and alone: the same bits."""
    m, N, K = [48 + 16 * (g % 5) for g in range(40)], 528, 784
    dy, _ = random_columns(m, N, 500, COMPACT)
    x, _ = random_columns(m, K, 600, COMPACT)
    dw = torch.empty(40, N, K, device="cuda")
    abi.nvfp4_group_wgrad(dy, x, m, dw)
    for g in (0, 17, 39):
        o, r = sum(m[:g]), m[g]
        one = [abi.matrix(q["data"][n * o // 2:n * (o + r) // 2].clone(), q["scale"][n * o // 16:n * (o + r) // 16].clone(),
                          q["s2"][g * n:(g + 1) * n].clone()) for q, n in ((dy, N), (x, K))]
        alone = torch.empty(1, N, K, device="cuda")
        abi.nvfp4_group_wgrad(*one, [r], alone)
        assert torch.equal(alone[0], dw[g])
