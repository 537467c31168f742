"""Low-rank adapters beside a shared NVFP4 projection against fp64."""
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


def case(rows, K, N, R, L, ids, seed, layout=COMPACT):
    g = torch.Generator().manual_seed(seed)
    x, xv = random_matrix(rows, K, seed, layout)
    w, wv = random_matrix(N, K, seed + 1, layout)
    x["s2"] *= 2.0 ** -6
    xv = xv * 2.0 ** -6
    xb = torch.randn(rows, K, generator=g).to(torch.bfloat16)
    a = (torch.randn(L, R, K, generator=g) * K ** -0.5).to(torch.bfloat16)
    b = torch.randn(L, N, R, generator=g).to(torch.bfloat16)
    f = torch.rand(L, generator=g) * 2
    return dict(x=x, xv=xv, w=w, wv=wv, xb=xb.cuda(), a=a.cuda(), b=b.cuda(), f=f.cuda(),
                ids=torch.tensor(ids, dtype=torch.int32).cuda())


def reference(c):
    """fp64, and the bound: the projection's; K roundings of 2^-24 in u's fp32
    sums (truncated MMA steps of 16: at most K / 4 cuts of 2^-23), R + 2 in
    the second sum and one in the last addition."""
    p, lim = product(c["xv"], c["wv"])
    xb, a, b, f = (c[k].double().cpu() for k in ("xb", "a", "b", "f"))
    K, R, L = xb.shape[1], a.shape[1], a.shape[0]
    for t, i in enumerate(c["ids"].cpu().tolist()):
        if 0 <= i < L:
            u = f[i] * (a[i] @ xb[t])
            lu = (K / 4 + 4) * 2.0 ** -23 * f[i] * (a[i].abs() @ xb[t].abs())
            y = b[i] @ u
            s = b[i].abs() @ u.abs()
            lim[t] += b[i].abs() @ lu + (R + 3) * 2.0 ** -24 * (s + p[t].abs())
            p[t] += y
    return p, lim


def run(c, dtype=torch.bfloat16, extra=2):
    rows, N, R = c["xb"].shape[0], c["b"].shape[1], c["a"].shape[1]
    buf = torch.full((rows + extra, N), 7.0, dtype=dtype, device="cuda")
    ws = abi.alloc_adapter_workspace(rows, R)
    ws.fill_(0xFF)  # NaN: what the second half reads has to be written by the first
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    abi.nvfp4_adapter_gemm(c["xb"], c["x"], c["w"], c["a"], c["b"], c["f"], c["ids"], buf[:rows], ws, st)
    assert bool((buf[rows:] == 7.0).all())
    return buf[:rows], int(st.item())


def spread(rows, L, kind):
    if kind == "one":
        return [L - 1] * rows
    if kind == "each":
        return [i % L for i in range(rows)]
    if kind == "runs":
        return [(i // 37) % (L + 1) - 1 for i in range(rows)]
    if kind == "none":
        return [-1] * rows
    return [(i * 7919) % (L + 1) - 1 for i in range(rows)]


@pytest.mark.parametrize("kind", ["one", "each", "runs", "none", "mixed"])
@pytest.mark.parametrize("rows,K,N,R,L", [(1, 64, 16, 8, 1), (17, 256, 144, 16, 5), (64, 1024, 256, 24, 64), (300, 528, 272, 64, 9),
                                          (33, 4096, 128, 40, 3)])
def test_adapters(rows, K, N, R, L, kind):
    c = case(rows, K, N, R, L, spread(rows, L, kind), rows + K)
    y, st = run(c)
    assert st == 0
    check(y, *reference(c), f"{rows} {K} {N} {R} {L} {kind}")


@pytest.mark.parametrize("rows,K,N,L", [(238, 512, 1760, 20), (100, 256, 4096, 7), (600, 1024, 8192, 3), (37, 64, 8192, 37)])
@pytest.mark.parametrize("kind", ["each", "runs", "none"])
def test_many_small_tiles_a_cta(rows, K, N, L, kind):
    """More tiles than SMs, of fewer rows than the columns that two accumulators share."""
    c = case(rows, K, N, 16, L, spread(rows, L, kind), rows + N)
    for _ in range(3):
        y, st = run(c)
        assert st == 0
    check(y, *reference(c), f"{rows} {K} {N} {L} {kind}")


@pytest.mark.parametrize("R", [8, 32, 48, 56, 64])
def test_fp32_and_every_rank(R):
    c = case(40, 320, 48, R, 4, spread(40, 4, "mixed"), R)
    y, st = run(c, torch.float32)
    assert st == 0
    check(y, *reference(c), f"rank {R}")


def test_prompts_of_many_rows():
    """More than 32 rows a SM: the wider token blocks."""
    rows = 148 * 32 + 5
    c = case(rows, 128, 64, 16, 6, [(i // 611) % 7 - 1 for i in range(rows)], 3)
    y, st = run(c)
    assert st == 0
    check(y, *reference(c))


def test_tiled_operands():
    c = case(256, 256, 256, 16, 3, spread(256, 3, "runs"), 4, TILED)
    y, st = run(c)
    assert st == 0
    check(y, *reference(c))


def test_ids_outside_the_adapters():
    """Reported, and such a token gets no adapter."""
    ids = [0, 5, -2, 1, 2 ** 31 - 1, -2 ** 31, 2, -1]
    c = case(8, 128, 48, 8, 3, ids, 5)
    y, st = run(c)
    assert st == abi.NVFP4_ERR_ROUTING
    check(y, *reference(c))


def test_no_adapter_equals_the_projection():
    c = case(50, 256, 160, 16, 2, [-1] * 50, 6)
    y, st = run(c, torch.float32)
    z = torch.empty_like(y)
    abi.nvfp4_group_gemm(c["x"], [50], c["w"], z)
    assert st == 0 and torch.equal(y, z)


def test_no_adapters_at_all():
    c = case(9, 64, 16, 8, 1, [-1] * 9, 7)
    c["a"], c["b"], c["f"] = c["a"][:0], c["b"][:0], c["f"][:0]
    y, st = run(c)
    assert st == 0
    check(y, *product(c["xv"], c["wv"]))


def test_token_does_not_depend_on_its_neighbours():
    """The same bits alone and among others, whatever they use."""
    c = case(70, 512, 96, 16, 8, spread(70, 8, "each"), 8)
    y, _ = run(c, torch.float32)
    for t in (0, 13, 69):
        one = dict(c, xb=c["xb"][t:t + 1].contiguous(), ids=c["ids"][t:t + 1].contiguous(),
                   x=abi.matrix(*(c["x"][k][t:t + 1].contiguous() for k in ("data", "scale", "s2"))))
        z, _ = run(one, torch.float32)
        assert torch.equal(y[t:t + 1], z)
    again, _ = run(c, torch.float32)
    assert torch.equal(y, again)


def test_graph_replays_with_other_ids():
    c = case(20, 256, 64, 16, 4, spread(20, 4, "each"), 9)
    y = torch.empty(20, 64, device="cuda")
    ws = abi.alloc_adapter_workspace(20, 16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        abi.nvfp4_adapter_gemm(c["xb"], c["x"], c["w"], c["a"], c["b"], c["f"], c["ids"], y, ws, st)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for kind in ("one", "none", "mixed"):
        c["ids"].copy_(torch.tensor(spread(20, 4, kind), dtype=torch.int32))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        check(y, *reference(c), kind)


def neighbours_case(seed, rows=70, L=5, K=256, N=96, R=40, kind="each"):
    return case(rows, K, N, R, L, spread(rows, L, kind), seed)


def non_finite(part, bad, kind, dtype):
    """Tokens of the other adapters, or of none, keep the bits that they have beside a
    finite adapter; the adapter's own tokens get what the formula gives."""
    c = neighbours_case(40, kind=kind)
    clean, _ = run(c, dtype)
    i, n, r, k = 2, 37, 35, 100
    own = c["ids"].cpu() == i
    assert 3 < int(own.sum()) < 40
    d = dict(c)
    d[part] = c[part].clone()
    d[part][{"a": (i, r, k), "b": (i, n, r), "f": (i,)}[part]] = bad
    y, st = run(d, dtype)
    assert st == 0
    assert torch.equal(y[~own.cuda()], clean[~own.cuda()])
    # the formula in fp64: which results are infinite (and with which sign), which are NaN
    p, _ = product(c["xv"], c["wv"])
    a, b, f, xb = (d[q].double().cpu() for q in ("a", "b", "f", "xb"))
    want = p[own] + (f[i] * (xb[own] @ a[i].t())) @ b[i].t()
    got = y.cpu()[own].double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(want)) and torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    # its finite results are those of the finite adapter: the changed element of b is not in them
    keep = torch.arange(y.shape[1]) != n
    if part == "b":
        ref, lim = reference(c)
        check(y.cpu()[own][:, keep], ref[own][:, keep], lim[own][:, keep], "finite features")


BAD = [float("inf"), float("-inf"), float("nan")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["each", "mixed"])
@pytest.mark.parametrize("bad", BAD)
def test_non_finite_b_stays_in_its_tokens(bad, kind, dtype):
    non_finite("b", bad, kind, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["each", "mixed"])
@pytest.mark.parametrize("part", ["a", "f"])
@pytest.mark.parametrize("bad", BAD)
def test_non_finite_u(part, bad, kind, dtype):
    """An infinity or NaN in a or in the factor, so in u."""
    non_finite(part, bad, kind, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["one", "mixed"])
def test_u_above_the_largest_bf16(kind, dtype):
    """u = 2^127 (2 - 2^-9): finite in fp32, and above 2^127 (2 - 2^-8), from where bf16
    rounds to infinity. The tokens beside it, of the same adapter too, keep their bits."""
    c = case(9, 64, 48, 8, 2, spread(9, 2, kind), 11)
    t = 4
    i = int(c["ids"][t])
    assert i >= 0
    c["b"] *= 2.0 ** -100
    c["xb"][:, 5] = 0.5
    c["a"][i, 3, 5] = 2.0 ** 63
    c["f"][i] = 2 - 2.0 ** -9
    base, _ = run(c, dtype)
    c["xb"][t] = 0
    c["xb"][t, 5] = 2.0 ** 64
    y, st = run(c, dtype)
    assert st == 0
    u = c["f"][i].double() * 2.0 ** 127
    assert float(torch.finfo(torch.bfloat16).max) < float(u) < float(torch.finfo(torch.float32).max)
    check(y, *reference(c), kind)
    rest = [r for r in range(9) if r != t]
    assert torch.equal(y[rest], base[rest])


def part_of(c, lo, hi):
    return dict(c, xb=c["xb"][lo:hi].clone(), ids=c["ids"][lo:hi].clone(),
                x=abi.matrix(*(c["x"][k][lo:hi].clone() for k in ("data", "scale", "s2"))))


@pytest.mark.parametrize("K", [1024, 4096, 7168])
def test_token_does_not_depend_on_the_size_of_the_call(K):
    """The same bits among 4741 rows, 70, 17 and alone, with 8 adapters or 33 loaded: the first half's
    sum over K has one order, however many CTAs share it."""
    rows = 148 * 32 + 5
    c = case(rows, K, 96, 16, 8, spread(rows, 8, "mixed"), 12)
    y, st = run(c, torch.float32)
    assert st == 0
    for lo, hi in ((0, 70), (3, 20), (13, 14), (4740, 4741)):
        z, _ = run(part_of(c, lo, hi), torch.float32)
        assert torch.equal(y[lo:hi], z), (lo, hi)
    more = part_of(c, 0, 70)
    for k in ("a", "b", "f"):
        more[k] = torch.cat([c[k], c[k], c[k], c[k], c[k][:1]])
    z, _ = run(more, torch.float32)
    assert torch.equal(y[:70], z)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_precision_where_the_adapter_cancels_the_projection(dtype):
    """b = -p / u rounded to bf16, so that y is what that rounding leaves, 2^-9 of p or less. u is one product, f a x:
    a and x of 8 bits, f of 24, rounded once (2^-24). For a bf16 y two bf16 terms of u are taken,
    within 2^-17 of it, for an fp32 y three, within 2^-25. Their products with b are exact, their sum is cut
    to 24 bits at most four times (2^-23 each), and one addition to p follows."""
    rows, K, N, R = 24, 64, 96, 8
    c = case(rows, K, N, R, rows, list(range(rows)), 13)
    c["xb"][:, 1:] = 0
    c["xb"][:, 0] = 1.0 + (torch.arange(rows) % 7 / 8.0).cuda()
    c["a"].zero_()
    c["a"][:, 0, 0] = 1.3125
    c["f"] = 0.5 + torch.rand(rows, generator=torch.Generator().manual_seed(14)).cuda()
    p, lim = product(c["xv"], c["wv"])
    u = c["f"].double().cpu() * 1.3125 * c["xb"][:, 0].double().cpu()
    b = (-p / u[:, None]).to(torch.bfloat16)
    c["b"].zero_()
    c["b"][:, :, 0] = b.cuda()
    d = b.double() * u[:, None]
    terms = 2.0 ** -17 if dtype == torch.bfloat16 else 2.0 ** -25
    y, st = run(c, dtype)
    assert st == 0
    want = p + d
    assert float(want.abs().max()) < 2.0 ** -8 * float(p.abs().max())
    check(y, want, lim + (terms + 2.0 ** -24 + 4 * 2.0 ** -23) * d.abs() + 2.0 ** -24 * want.abs())


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (129, 16), (7, 1008), (131, 176)])
def test_scales_that_end_inside_a_word(rows, K):
    """The projection's row-major scales end 1, 2 or 3 bytes into an aligned word (rows K / 16 bytes)."""
    assert rows * (K // 16) % 4
    c = case(rows, K, 48, 8, 3, spread(rows, 3, "mixed"), rows + K)
    y, st = run(c, torch.float32)
    assert st == 0
    check(y, *reference(c))


def test_two_streams_at_once():
    """Decode steps and prompts on two streams, a workspace each: the bits of one call after the other."""
    if os.environ.get("NVFP4RS_LIBRARY", "").endswith("_debug.so"):
        pytest.skip("the bounds-checked build keeps one table of ranges: one call at a time")
    cs = [case(64, 1024, 512, 16, 64, spread(64, 64, "each"), 15), case(3000, 1024, 512, 32, 5, spread(3000, 5, "runs"), 16)]
    want = [run(c)[0].clone() for c in cs]
    ys = [torch.empty_like(w) for w in want]
    ws = [abi.alloc_adapter_workspace(c["xb"].shape[0], c["a"].shape[1]) for c in cs]
    st = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(50):
        for c, y, w, s, stream in zip(cs, ys, ws, st, streams):
            abi.nvfp4_adapter_gemm(c["xb"], c["x"], c["w"], c["a"], c["b"], c["f"], c["ids"], y, w, s, stream=stream)
    torch.cuda.synchronize()
    for y, w, s in zip(ys, want, st):
        assert int(s.item()) == 0 and torch.equal(y, w)
