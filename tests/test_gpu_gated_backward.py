"""The gated product's gradient against fp64 and against differences, and its
amax against the grouped amax of the result, bit for bit."""
import pytest
import torch

from nvfp4_row_scaled_b200 import abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_row_scaled_b200.build import build_library
    build_library()
    abi.lib()


def inputs(rows, F, seed, spread=4.0):
    g = torch.Generator().manual_seed(seed)
    dh = torch.randn(rows, F, generator=g) * torch.exp2(torch.rand(rows, 1, generator=g) * 8 - 8)
    gu = torch.randn(rows, 2 * F, generator=g) * spread
    if rows > 3:
        dh[1] = 0
        gu[2] = 0
        gu[3, :F] = 120.0 * (torch.arange(F) % 2 * 2 - 1)  # sigmoid at 0 and at 1
    return dh.to(torch.bfloat16).cuda(), gu.to(torch.bfloat16).cuda()


def reference(dh, gu):
    """fp64 gradient and the bound of the fp32 formula: e^-g to 2 ulp plus its
    rounded argument (|g| 2^-24), the quotient 2 ulp, four products, and the
    factor 1 + g (1 - s), whose terms cancel near g = -1.28: its error is at
    most (1 + |g|) parts of the relative error."""
    F = dh.shape[1]
    dh, g, u = dh.double().cpu(), gu[:, :F].double().cpu(), gu[:, F:].double().cpu()
    s = torch.sigmoid(g)
    dg = dh * u * s * (1 + g * torch.sigmoid(-g))
    du = dh * g * s
    eps = (12 + g.abs()) * 2.0 ** -23
    return (torch.cat([dg, du], 1),
            torch.cat([2 * eps * (dh * u * s).abs() * (1 + g.abs()), eps * du.abs()], 1))


SHAPES = [([16], 16), ([64], 256), ([16, 0, 48, 32], 272), ([128, 256], 2048), ([16] * 9, 528), ([1040], 512),
          ([48, 80], 8192), ([32], 65536)]


@pytest.mark.parametrize("m,F", SHAPES)
def test_gradient_and_amax(m, F):
    rows, E = sum(m), len(m)
    dh, gu = inputs(rows, F, 1)
    buf = torch.full((rows + 2, 2 * F), 7.0, dtype=torch.bfloat16, device="cuda")
    d = buf[:rows]
    ra = torch.full((rows + 2,), 7.0, device="cuda")
    ca = torch.full((E * 2 * F,), 7.0, device="cuda")
    abi.nvfp4_group_gated_backward(dh, gu, m, d, ra[:rows], ca)
    want, lim = reference(dh, gu)
    got = d.double().cpu()
    # below 2^-126 the factors of the fp32 formula leave its normal range
    assert bool(((got - want).abs() <= lim + 2.0 ** -8 * (want.abs() + lim) + 1e-36).all())
    assert bool((buf[rows:] == 7.0).all()) and bool((ra[rows:] == 7.0).all())
    wr, wc = abi.alloc_amax(rows, 2 * F, E)
    abi.nvfp4_group_amax(d.contiguous(), m, wr, wc)
    assert torch.equal(ra[:rows], wr) and torch.equal(ca, wc)


def test_parts_can_be_left_out_and_in_place():
    m, F = [48, 16], 144
    dh, gu = inputs(64, F, 2)
    d = torch.empty_like(gu)
    ra, ca = abi.alloc_amax(64, 2 * F, 2)
    abi.nvfp4_group_gated_backward(dh, gu, m, d, ra, ca)
    d2, ra2 = torch.empty_like(gu), torch.empty_like(ra)
    abi.nvfp4_group_gated_backward(dh, gu, m, d2, row_amax=ra2)
    ca2 = torch.empty_like(ca)
    d3 = torch.empty_like(gu)
    abi.nvfp4_group_gated_backward(dh, gu, m, d3, col_amax=ca2)
    abi.nvfp4_group_gated_backward(dh, gu, m, gu)
    assert torch.equal(d, d2) and torch.equal(d, d3) and torch.equal(d, gu)
    assert torch.equal(ra, ra2) and torch.equal(ca, ca2)


def test_against_differences():
    """(h(p + e) - h(p - e)) / 2e in fp64 at the saved pre-activations: the
    difference's own error is e^2/6 |h'''| <= e^2, the kernel's the test's above."""
    rows, F, e = 32, 64, 1e-4
    dh, gu = inputs(rows, F, 3, spread=2.0)
    d = torch.empty_like(gu)
    abi.nvfp4_group_gated_backward(dh, gu, [rows], d)
    p = gu.double().cpu()

    def h(q):
        return q[:, :F] * torch.sigmoid(q[:, :F]) * q[:, F:] * dh.double().cpu()
    for half in (0, 1):
        q = torch.zeros_like(p)
        q[:, half * F:(half + 1) * F] = e
        num = (h(p + q) - h(p - q)) / (2 * e)
        got = d[:, half * F:(half + 1) * F].double().cpu()
        _, lim = reference(dh, gu)
        lim = lim[:, half * F:(half + 1) * F]
        scale = dh.double().cpu().abs() * (1 + p[:, F:].abs())
        # fp64 cancellation in the difference: 2^-52 |h| / e, |h| <= scale |g|
        assert bool(((got - num).abs() <= lim + 2.0 ** -8 * num.abs() * 1.01 + scale * (e * e + 130 * 2.0 ** -52 / e) + 1e-36).all())


def test_graphsafe_equals_host_split_and_replays():
    F, E, cap = 144, 3, 160
    dh, gu = inputs(cap, F, 4)
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    fd, offs = abi.routing_tensors([64, 0, 96], 2 * F)
    d, ra, ca = torch.empty_like(gu), torch.empty(cap, device="cuda"), torch.empty(E * 2 * F, device="cuda")
    abi.nvfp4_group_gated_backward_graphsafe(dh, gu, fd, offs, d, st, ra, ca)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.nvfp4_group_gated_backward_graphsafe(dh, gu, fd, offs, d, st, ra, ca)
    for m in ([64, 0, 96], [16, 16, 0], [0, 0, 0], [160, 0, 0]):
        f2, o2 = abi.routing_tensors(m, 2 * F)
        fd.copy_(f2)
        offs.copy_(o2)
        d.fill_(7.0)
        ra.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        n = sum(m)
        assert bool((d[n:] == 7.0).all()) and bool((ra[n:] == 7.0).all())
        dw, wr, wc = torch.empty_like(gu[:n]), torch.empty(n, device="cuda"), torch.empty(E * 2 * F, device="cuda")
        abi.nvfp4_group_gated_backward(dh[:n].contiguous(), gu[:n].contiguous(), m, dw, wr, wc)
        assert torch.equal(d[:n], dw) and torch.equal(ra[:n], wr) and torch.equal(ca, wc)
    f2, o2 = abi.routing_tensors([8, 8, 0], 2 * F)
    fd.copy_(f2)
    offs.copy_(o2)
    d.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == abi.NVFP4_ERR_UNSUPPORTED and bool((d == 7.0).all())


def test_every_gate():
    """Gates at which e^-g is above 2^126 or infinite and e^g below 2^-126, dh and up large
    and small: both gradients to the formula's bound and half a step, with no absolute allowance but
    bf16's smallest steps."""
    gate = torch.cat([torch.tensor([-1400.0, -300.0, -172.0, -150.0, -104.0, -103.0, -90.0, -88.5, -88.0, -87.5, -87.0, -30.0, -1.0,
                                    -0.0, 1e-30, 0.5, 20.0, 87.0, 87.5, 88.5, 89.0, 104.0, 1400.0, 3e38]),
                      torch.linspace(-172, 172, 104)])
    up = torch.tensor([2.0 ** 100, 1.0, 2.0 ** 40, 2.0 ** -40])
    dh0 = torch.tensor([2.0 ** 20, 1.0, 2.0 ** 80, 2.0 ** 30])
    rows, F = 16, gate.numel()
    gu = torch.cat([gate.expand(rows, F), up.repeat(4)[:, None].expand(rows, F)], 1).to(torch.bfloat16).contiguous().cuda()
    dh = dh0.repeat(4)[:, None].expand(rows, F).to(torch.bfloat16).contiguous().cuda()
    dh[:, 23] = 2.0 ** -10  # beside the gate of 3e38: products that fit
    gu[:, F + 23] = 2.0 ** -10
    d = torch.empty_like(gu)
    abi.nvfp4_group_gated_backward(dh, gu, [rows], d)
    want, lim = reference(dh, gu)
    got = d.double().cpu()
    err, room = (got - want).abs(), lim + 2.0 ** -8 * (want.abs() + lim) + 2.0 ** -134
    bad = ~(err <= room)
    assert not bool(bad.any()), (gu.cpu()[:, :F].repeat(1, 2)[bad], got[bad], want[bad])


@pytest.mark.parametrize("m,F", [([16], 16), ([48, 80], 8192), ([16, 0, 48, 32], 272), ([32], 65536), ([16] * 37, 2048),
                                 ([4096, 16, 2064], 1024)])
def test_in_place(m, F):
    """d_gate_up written over gate_up: the same bits as beside it, over clusters of 1 to 8 CTAs
    and tiles that hold several groups, host-split and graph-safe."""
    rows, E = sum(m), len(m)
    dh, gu = inputs(rows, F, 6)
    d, (ra, ca) = torch.empty_like(gu), abi.alloc_amax(rows, 2 * F, E)
    abi.nvfp4_group_gated_backward(dh, gu, m, d, ra, ca)
    fd, offs = abi.routing_tensors(m, 2 * F)
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    for graphsafe in (False, True):
        p = gu.clone()
        ra2, ca2 = abi.alloc_amax(rows, 2 * F, E)
        if graphsafe:
            abi.nvfp4_group_gated_backward_graphsafe(dh, p, fd, offs, p, st, ra2, ca2)
            assert int(st.item()) == 0
        else:
            abi.nvfp4_group_gated_backward(dh, p, m, p, ra2, ca2)
        assert torch.equal(p, d) and torch.equal(ra2, ra) and torch.equal(ca2, ca)
