"""The casts and the products together, as a training step and a serving step of
grouped experts use them: every product against fp64 on the values of the bytes
that the casts wrote; the step as one CUDA graph over changing routings; and the
gradients of the whole block against differences."""
import pytest
import torch

from nvfp4_row_scaled_b200 import abi

from .products import check, product, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_row_scaled_b200.build import build_library
    build_library()
    abi.lib()


def cast(x, m):
    """Both directions of the grouped cast of x [rows, K]."""
    rows, K, E = x.shape[0], x.shape[1], len(m)
    ra, ca = abi.alloc_amax(rows, K, E)
    out = abi.alloc_outputs(rows, K, E)
    abi.nvfp4_group_amax(x, m, ra, ca)
    abi.nvfp4_group_cast(x, m, ra, ca, out)
    return out


def row_values(out, K):
    return values(out["row_data"].view(-1, K // 2), out["row_scale"].view(-1, K // 16), out["row_s2"], K)


def col_values(out, m, K):
    """Each group's transpose [K, m_g]."""
    res, o = [], 0
    for g, r in enumerate(m):
        res.append(values(out["col_data"][K * o // 2:K * (o + r) // 2].view(K, r // 2),
                          out["col_scale"][K * o // 16:K * (o + r) // 16].view(K, r // 16), out["col_s2"][g * K:(g + 1) * K], r))
        o += r
    return res


def grouped(xv, m, ws):
    p, b, o = [], [], 0
    for r, w in zip(m, ws):
        q, lim = product(xv[o:o + r], w)
        p.append(q)
        b.append(lim)
        o += r
    return torch.cat(p), torch.cat(b)


def bf16(*shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("m,K,F", [([16, 0, 48, 128], 128, 64), ([128, 256], 256, 128), ([32], 144, 80)])
def test_training_step(m, K, F):
    rows, E = sum(m), len(m)
    g = torch.Generator().manual_seed(rows + K)
    x = torch.randn(rows, K, generator=g).to(torch.bfloat16).cuda()
    w1 = (torch.randn(E * 2 * F, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda()
    w2 = (torch.randn(E * K, F, generator=g) * F ** -0.5).to(torch.bfloat16).cuda()
    dy = torch.randn(rows, K, generator=g).to(torch.bfloat16).cuda()
    xq, w1q, w2q, dyq = cast(x, m), cast(w1, [2 * F] * E), cast(w2, [K] * E), cast(dy, m)

    h, gu = bf16(rows, F), bf16(rows, 2 * F)
    abi.nvfp4_group_gated_gemm(abi.row_matrix(xq), m, abi.row_matrix(w1q), h, gate_up=gu)
    p, lim = grouped(row_values(xq, K), m, row_values(w1q, K).split(2 * F))
    check(gu, p, lim, "gate_up")

    hq = cast(h, m)
    y = bf16(rows, K)
    abi.nvfp4_group_gemm(abi.row_matrix(hq), m, abi.row_matrix(w2q), y)
    check(y, *grouped(row_values(hq, F), m, row_values(w2q, F).split(K)), "y")

    dh = bf16(rows, F)
    abi.nvfp4_group_gemm(abi.row_matrix(dyq), m, abi.col_matrix(w2q), dh)
    check(dh, *grouped(row_values(dyq, K), m, col_values(w2q, [K] * E, F)), "dh")
    dw2 = torch.empty(E, K, F, device="cuda")
    abi.nvfp4_group_wgrad(abi.col_matrix(dyq), abi.col_matrix(hq), m, dw2)
    for e, (a, b) in enumerate(zip(col_values(dyq, m, K), col_values(hq, m, F))):
        check(dw2[e], *product(a, b), f"dw2 {e}")

    dgu = bf16(rows, 2 * F)
    ra, ca = abi.alloc_amax(rows, 2 * F, E)
    abi.nvfp4_group_gated_backward(dh, gu, m, dgu, ra, ca)
    gq = abi.alloc_outputs(rows, 2 * F, E)
    abi.nvfp4_group_cast(dgu, m, ra, ca, gq)
    for k, v in cast(dgu, m).items():  # the amax of the fused pass is the grouped amax
        assert torch.equal(gq[k], v), k
    dx = bf16(rows, K)
    abi.nvfp4_group_gemm(abi.row_matrix(gq), m, abi.col_matrix(w1q), dx)
    check(dx, *grouped(row_values(gq, 2 * F), m, col_values(w1q, [2 * F] * E, K)), "dx")
    dw1 = torch.empty(E, 2 * F, K, device="cuda")
    abi.nvfp4_group_wgrad(abi.col_matrix(gq), abi.col_matrix(xq), m, dw1)
    for e, (a, b) in enumerate(zip(col_values(gq, m, 2 * F), col_values(xq, m, K))):
        check(dw1[e], *product(a, b), f"dw1 {e}")


def test_block_gradients_against_differences():
    """d(sum(h c)) / dx and / dW of the gated block on operands that NVFP4 holds
    exactly (to the rounding of its decode factor), so that only the gradient's own cast is inexact: its products are
    compared with differences of the fp64 block within half an E2M1 step (1/6 of
    a block's largest value at most: steps of 2 from 4 to 6, so half a step is 1 of
    6) of d(gate|up), summed over the contraction."""
    m, K, F = [32], 32, 16
    g = torch.Generator().manual_seed(5)
    # +-{1, 1.5, 2, 3}: with amax 6 in every block the cast is exact
    def exact(rows, cols, scale):
        v = torch.tensor([1.0, 1.5, 2.0, 3.0, 6.0])[torch.randint(0, 5, (rows, cols), generator=g)]
        v = v * (torch.randint(0, 2, (rows, cols), generator=g) * 2 - 1)
        v[::16, :] = 6.0
        v[:, ::16] = 6.0
        return (v * scale).to(torch.bfloat16).cuda()
    x, w = exact(32, K, 2.0 ** -5), exact(2 * F, K, 2.0 ** -2)
    xq, wq = cast(x, m), cast(w, [2 * F])
    # exact but for the decode factor: a code times 448 times fl(amax / 2688), one rounding of 2^-24
    for got, want in ((row_values(xq, K), x.double().cpu()), (row_values(wq, K), w.double().cpu())):
        assert bool(((got - want).abs() <= 2.0 ** -24 * want.abs()).all())
    h, gu = bf16(32, F), bf16(32, 2 * F)
    abi.nvfp4_group_gated_gemm(abi.row_matrix(xq), m, abi.row_matrix(wq), h, gate_up=gu)
    c = torch.randn(32, F, generator=g).to(torch.bfloat16).cuda()
    dgu, (ra, ca) = bf16(32, 2 * F), abi.alloc_amax(32, 2 * F, 1)
    abi.nvfp4_group_gated_backward(c, gu, m, dgu, ra, ca)
    gq = abi.alloc_outputs(32, 2 * F, 1)
    abi.nvfp4_group_cast(dgu, m, ra, ca, gq)
    dx, dw = torch.empty(32, K, device="cuda"), torch.empty(1, 2 * F, K, device="cuda")
    abi.nvfp4_group_gemm(abi.row_matrix(gq), m, abi.col_matrix(wq), dx)
    abi.nvfp4_group_wgrad(abi.col_matrix(gq), abi.col_matrix(xq), m, dw)

    xv, wv, cv = x.double().cpu(), w.double().cpu(), c.double().cpu()

    def loss(a, b):
        p = a @ b.t()
        return (p[:, :F] * torch.sigmoid(p[:, :F]) * p[:, F:] * cv).sum()
    a, b = xv.clone().requires_grad_(True), wv.clone().requires_grad_(True)
    loss(a, b).backward()
    e = 1e-6
    for _ in range(20):  # the reference itself against differences
        i, j = int(torch.randint(0, 32, (1,), generator=g)), int(torch.randint(0, K, (1,), generator=g))
        for t, grad in ((0, a.grad), (1, b.grad)):
            up, dn = [xv.clone(), wv.clone()], [xv.clone(), wv.clone()]
            up[t][i, j] += e
            dn[t][i, j] -= e
            num = (loss(*up) - loss(*dn)) / (2 * e)
            assert abs(float(num - grad[i, j])) <= 1e-6 * (1 + abs(float(grad[i, j])))
    # error of the cast of d(gate|up): at most 1/6 of its row's (column's) largest value an
    # element, plus the bf16 roundings of it and of the saved pre-activations (2^-7 of it at most here)
    d = dgu.double().cpu().abs()
    lim_x = (1 / 6 + 2.0 ** -6) * d.amax(1, keepdim=True) * wv.abs().sum(0)[None, :]
    lim_w = (1 / 6 + 2.0 ** -6) * d.amax(0)[:, None] * xv.abs().sum(0)[None, :]
    assert bool(((dx.double().cpu() - a.grad).abs() <= lim_x).all())
    assert bool(((dw[0].double().cpu() - b.grad).abs() <= lim_w).all())
    # and it points the same way
    for got, want in ((dx, a.grad), (dw[0], b.grad)):
        got = got.double().cpu()
        assert float((got * want).sum() / (got.norm() * want.norm())) > 0.98


def test_step_as_one_graph_over_routings():
    """Casts and products captured once with device routing; each replay equals the
    host-split calls on that routing."""
    K, F, E, cap = 128, 64, 3, 256
    g = torch.Generator().manual_seed(9)
    x = torch.randn(cap, K, generator=g).to(torch.bfloat16).cuda()
    w1 = (torch.randn(E * 2 * F, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda()
    dh = torch.randn(cap, F, generator=g).to(torch.bfloat16).cuda()
    w1q = cast(w1, [2 * F] * E)
    fd, ox = abi.routing_tensors([64, 64, 128], K)
    _, og = abi.routing_tensors([64, 64, 128], 2 * F)
    st = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(7)]
    xq, gq = abi.alloc_outputs(cap, K, E), abi.alloc_outputs(cap, 2 * F, E)
    ra, ca = abi.alloc_amax(cap, K, E)
    rg, cg = abi.alloc_amax(cap, 2 * F, E)
    h, gu, dgu, dx = bf16(cap, F), bf16(cap, 2 * F), bf16(cap, 2 * F), bf16(cap, K)
    dw = torch.empty(E, 2 * F, K, device="cuda")

    def step():
        abi.nvfp4_group_amax_graphsafe(x, fd, ox, ra, ca, st[0])
        abi.nvfp4_group_cast_graphsafe(x, fd, ox, ra, ca, xq, st[1])
        abi.nvfp4_group_gated_gemm_graphsafe(abi.row_matrix(xq), fd, ox, abi.row_matrix(w1q), h, st[2], gate_up=gu)
        abi.nvfp4_group_gated_backward_graphsafe(dh, gu, fd, og, dgu, st[3], rg, cg)
        abi.nvfp4_group_cast_graphsafe(dgu, fd, og, rg, cg, gq, st[4])
        abi.nvfp4_group_gemm_graphsafe(abi.row_matrix(gq), fd, og, abi.col_matrix(w1q), dx, st[5])
        abi.nvfp4_group_wgrad_graphsafe(abi.col_matrix(gq), abi.col_matrix(xq), cap, fd, ox, dw, st[6])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for m in ([64, 64, 128], [16, 0, 48], [0, 0, 256], [0, 0, 0]):
        for t, K_ in ((ox, K), (og, 2 * F)):
            f2, o2 = abi.routing_tensors(m, K_)
            fd.copy_(f2)
            t.copy_(o2)
        for t in (h, gu, dgu, dx, dw):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(int(s.item()) == 0 for s in st)
        n = sum(m)
        for t in (h, gu, dgu, dx):
            assert bool((t[n:] == 7.0).all())
        xn, dhn = x[:n].contiguous(), dh[:n].contiguous()
        q = cast(xn, m)
        h2, gu2, dgu2, dx2 = bf16(n, F), bf16(n, 2 * F), bf16(n, 2 * F), bf16(n, K)
        abi.nvfp4_group_gated_gemm(abi.row_matrix(q), m, abi.row_matrix(w1q), h2, gate_up=gu2)
        r2, c2 = abi.alloc_amax(n, 2 * F, E)
        abi.nvfp4_group_gated_backward(dhn, gu2, m, dgu2, r2, c2)
        q2 = abi.alloc_outputs(n, 2 * F, E)
        abi.nvfp4_group_cast(dgu2, m, r2, c2, q2)
        abi.nvfp4_group_gemm(abi.row_matrix(q2), m, abi.col_matrix(w1q), dx2)
        dw2 = torch.empty_like(dw)
        abi.nvfp4_group_wgrad(abi.col_matrix(q2), abi.col_matrix(q), m, dw2)
        for a, b in ((h, h2), (gu, gu2), (dgu, dgu2), (dx, dx2)):
            assert torch.equal(a[:n], b)
        assert torch.equal(dw, dw2)


def test_serving_step():
    """A decode batch: one token a request, the shared projection with each
    request's adapter, then the experts with a token or two each."""
    T, K, F, E, R, L = 16, 256, 64, 8, 16, 5
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    wp = (torch.randn(K, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda()
    a = (torch.randn(L, R, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda()
    b = torch.randn(L, K, R, generator=g).to(torch.bfloat16).cuda()
    f = torch.rand(L, generator=g).cuda()
    ids = torch.tensor([i % (L + 1) - 1 for i in range(T)], dtype=torch.int32).cuda()
    xq, wq = cast(x, [T]), cast(wp, [K])
    y = bf16(T, K)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.nvfp4_adapter_gemm(x, abi.row_matrix(xq), abi.row_matrix(wq), a, b, f, ids, y, abi.alloc_adapter_workspace(T, R), st)
    assert int(st.item()) == 0
    want, lim = product(row_values(xq, K), row_values(wq, K))
    for t, i in enumerate(ids.tolist()):
        if i >= 0:
            ad, bd, xt, fi = a[i].double().cpu(), b[i].double().cpu(), x[t].double().cpu(), float(f[i])
            u = fi * (ad @ xt)
            lim[t] += bd.abs() @ ((K / 4 + 4) * 2.0 ** -23 * fi * (ad.abs() @ xt.abs())) + (R + 3) * 2.0 ** -16 * (bd.abs() @ u.abs())
            want[t] += bd @ u
    check(y, want, lim, "projection")
    # the experts: the tokens in the experts' order, 16-row padding for the cast only
    m = [1, 0, 2, 5, 0, 3, 4, 1]
    w1 = (torch.randn(E * 2 * F, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda()
    w1q, yq, h = cast(w1, [2 * F] * E), cast(y, [T]), bf16(T, F)
    abi.nvfp4_group_gated_gemm(abi.row_matrix(yq), m, abi.row_matrix(w1q), h)
    p, lim = grouped(row_values(yq, K), m, row_values(w1q, K).split(2 * F))
    gate, up = p[:, :F], p[:, F:]
    s = gate * torch.sigmoid(gate)
    check(h, s * up, 1.1 * lim[:, :F] * (up.abs() + lim[:, F:]) + s.abs() * lim[:, F:] +
          (8 + gate.abs()) * 2.0 ** -22 * (s * up).abs(), "h")
