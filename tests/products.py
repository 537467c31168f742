"""Shared pieces of the tests of the products: random NVFP4 operands, their
values in fp64 straight from the bytes, and the error bound of a product."""
import torch

from nvfp4_row_scaled_b200 import abi

TILED = abi.NVFP4_SCALE_TILED_128X4
COMPACT = abi.NVFP4_SCALE_COMPACT

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def tile_scales(s: torch.Tensor) -> torch.Tensor:
    """Row-major [rows, cols] block scales in 128x4 tiles, by index."""
    rows, cols = s.shape
    r = torch.arange(rows, device=s.device)[:, None]
    c = torch.arange(cols, device=s.device)[None, :]
    at = ((r // 128) * (cols // 4) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    out = torch.empty(rows * cols, dtype=s.dtype, device=s.device)
    out[at.reshape(-1)] = s.reshape(-1)
    return out.view(rows, cols)


def random_matrix(rows, cols, seed, layout=COMPACT, device="cuda"):
    """Codes of every value, block scales over eight octaves (zero among
    them), row factors over four (zero among them); and its fp64 values."""
    g = torch.Generator().manual_seed(seed)
    data = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    scale = torch.randint(0x18, 0x58, (rows, cols // 16), generator=g, dtype=torch.int32).to(torch.uint8)
    scale[torch.rand(rows, cols // 16, generator=g) < 0.02] = 0
    s2 = torch.exp2(torch.rand(rows, generator=g) * 4 - 6) if rows else torch.zeros(0)
    s2[torch.rand(rows, generator=g) < 0.02] = 0
    m = abi.matrix(data.to(device), (tile_scales(scale) if layout == TILED else scale).contiguous().to(device),
                   s2.to(device), layout)
    return m, values(data, scale, s2, cols)


def values(data, scale, s2, cols):
    """fp64 [rows, cols] of one matrix with row-major scales."""
    data, scale, s2 = data.cpu(), scale.cpu(), s2.cpu()
    rows = s2.numel()
    code = torch.stack([data & 15, data >> 4], -1).view(rows, cols)
    v = E2M1[code.long()]
    return v * scale.view(rows, cols // 16).view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * s2.double()[:, None]


def product(x, w):
    """x w^T in fp64, and its error bound in the products' fp32 sums: an
    instruction sums four blocks of 16 exact products and the running sum, each
    of the five cut to 24 bits at most at the size of the largest partial sum,
    which is at most sum |x||w|; then two fp32 roundings of the result."""
    k = x.shape[1]
    p, s = x @ w.t(), x.abs() @ w.abs().t()
    return p, 5 * ((k + 63) // 64) * 2.0 ** -23 * s + 2 * 2.0 ** -24 * p.abs()


def check(got, want, bound, what=""):
    """|got - want| <= bound + half a step of got's type, everywhere; nothing NaN."""
    half = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu()
    err = (got - want).abs()
    lim = bound + half * (want.abs() + bound) + 1e-38
    bad = ~(err <= lim)
    if bool(bad.any()):
        i = tuple(int(v[0]) for v in torch.nonzero(bad, as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {got[i]} want {want[i]} "
                             f"limit {lim[i]}")
