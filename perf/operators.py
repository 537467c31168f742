"""The operators that use the grouped row-scaled NVFP4 cast, as they are measured.

Five operators, each in a plain form (elementary torch operations in fp32,
rounded once at the end) and as the calls a user makes of the library:

  gemm      y_g = X_g W_g^T, the grouped product of two casts (forward and, with
            the column-wise cast of W, the gradient of the input)
  wgrad     dW_g = dY_g^T X_g from the two column-wise casts
  gated     h_g = silu(X_g Wgate_g^T) * (X_g Wup_g^T): both projections, the
            activation and the product
  gated_bwd the gradient of that product: d(gate|up) from dh, with its row and
            per-group column amax (the scale sources of its cast)
  adapter   y_t = x^_t W^T + s_a (x_t A_a^T) B_a^T with a = id_t: low-rank
            adapters of many requests beside one shared NVFP4 projection

A matrix in NVFP4 is a dict: data (two E2M1 codes a byte, the first in the low
nibble), scale (one E4M3 byte for 16 elements, row-major or in 128x4 tiles),
s2 (one fp32 factor a row). Its value is (e2m1 * e4m3) * s2.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through one projection: the smallest call, all latency
        {"name": "gemm_one_token", "op": "gemm", "groups": 1, "rows": 1, "K": 2048, "N": 2048, "unit": 1,
         "skew": 0.0, "idle": 0, "tiled": False, "routing": 0},
        # 8 experts, 16384 packed rows in 128-row units
        {"name": "gemm_8_experts", "op": "gemm", "groups": 8, "rows": 16384, "K": 2048, "N": 2048, "unit": 128,
         "skew": 0.0, "idle": 0, "tiled": True, "routing": 1},
        # input gradient over groups of any length (nothing padded), row-major scales
        {"name": "gemm_ragged_dgrad", "op": "gemm", "groups": 16, "rows": 5003, "K": 4096, "N": 7168, "unit": 1,
         "skew": 1.1, "idle": 2, "tiled": False, "routing": 2},
        # the down projection of the DeepSeek-V3 routing: 256 experts, 26 of them idle
        {"name": "gemm_dsv3_down", "op": "gemm", "groups": 256, "rows": 80768, "K": 2048, "N": 7168, "unit": 128,
         "skew": 1.1, "idle": 26, "tiled": True, "routing": 3},
        # serving step of 128 experts with a few tokens each: bound by the weights
        {"name": "gated_decode", "op": "gated", "groups": 128, "rows": 512, "K": 2048, "F": 1024, "unit": 1,
         "skew": 0.6, "idle": 5, "tiled": False, "save": False, "routing": 4},
        # the gated projections of the DeepSeek-V3 routing, pre-activations kept for the gradient
        {"name": "gated_dsv3", "op": "gated", "groups": 256, "rows": 80768, "K": 7168, "F": 2048, "unit": 128,
         "skew": 1.1, "idle": 26, "tiled": True, "save": True, "routing": 3},
        # gradient of the gated product, a small packed batch
        {"name": "gated_bwd_small", "op": "gated_bwd", "groups": 8, "rows": 1024, "F": 2048, "unit": 16,
         "skew": 0.0, "idle": 1, "routing": 5},
        # the same at the DeepSeek-V3 routing
        {"name": "gated_bwd_dsv3", "op": "gated_bwd", "groups": 256, "rows": 80768, "F": 2048, "unit": 128,
         "skew": 1.1, "idle": 26, "routing": 3},
        # weight gradient of 8 experts, groups padded to 16 rows only
        {"name": "wgrad_8_experts", "op": "wgrad", "groups": 8, "rows": 8208, "K": 2048, "N": 4096, "unit": 16,
         "skew": 0.5, "idle": 0, "tiled": False, "fp32": False, "routing": 6},
        # weight gradient kept in fp32 for many experts
        {"name": "wgrad_fp32", "op": "wgrad", "groups": 16, "rows": 8192, "K": 4096, "N": 2048, "unit": 128,
         "skew": 0.5, "idle": 2, "tiled": True, "fp32": True, "routing": 7},
        # a decode step: 64 requests, one token each, most with an adapter of their own
        {"name": "adapter_decode", "op": "adapter", "rows": 64, "K": 4096, "N": 4096, "rank": 16, "adapters": 64,
         "requests": 64, "tiled": False, "routing": 8},
        # prompts of a few requests of uneven length
        {"name": "adapter_prompts", "op": "adapter", "rows": 8192, "K": 7168, "N": 2048, "rank": 32, "adapters": 8,
         "requests": 13, "tiled": True, "routing": 9},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gated", "gated", "gated_bwd", "wgrad", "adapter", "adapter"])
    routing = rng.randrange(1 << 20)
    if op == "adapter":
        rows = _log(rng, 1, 8192)
        return {"op": op, "rows": rows, "K": 64 * _log(rng, 4, 112), "N": 16 * _log(rng, 16, 256),
                "rank": 8 * rng.randint(1, 8), "adapters": _log(rng, 1, 64), "requests": _log(rng, 1, min(rows, 64)),
                "tiled": False, "routing": routing}
    groups = _log(rng, 1, 64)
    if op == "wgrad":
        rows = 16 * _log(rng, 1, 512)
        return {"op": op, "groups": groups, "rows": rows, "K": 16 * _log(rng, 8, 256), "N": 16 * _log(rng, 8, 128),
                "unit": 16, "skew": rng.uniform(0, 1.2), "idle": rng.randrange(0, max(1, groups // 4)),
                "tiled": False, "fp32": rng.random() < 0.5, "routing": routing}
    if op == "gated_bwd":
        return {"op": op, "groups": groups, "rows": 16 * _log(rng, 1, 4096), "F": 16 * _log(rng, 4, 128), "unit": 16,
                "skew": rng.uniform(0, 1.2), "idle": rng.randrange(0, max(1, groups // 4)), "routing": routing}
    tiled = rng.random() < 0.5
    rows = 128 * _log(rng, 1, 128) if tiled else _log(rng, 1, 16384)
    c = {"op": op, "groups": groups, "rows": rows, "K": (128 if tiled else 32) * _log(rng, 2, 32 if tiled else 128),
         "unit": 128 if tiled else 1, "skew": rng.uniform(0, 1.2), "idle": rng.randrange(0, max(1, groups // 4)),
         "tiled": tiled, "routing": routing}
    if op == "gemm":
        c["N"] = 128 * _log(rng, 1, 32) if tiled else 16 * _log(rng, 4, 256)
    else:
        c["F"] = 128 * _log(rng, 1, 16) if tiled else 16 * _log(rng, 4, 128)
        c["save"] = rng.random() < 0.5
    return c


def _splits(case):
    """Rows of each group: `rows` dealt in whole units over a shuffled Zipf
    law of exponent `skew`, with `idle` groups left empty."""
    r = np.random.RandomState(case["routing"])
    E, unit = case["groups"], case["unit"]
    p = np.arange(1, E + 1, dtype=np.float64) ** -case["skew"]
    r.shuffle(p)
    p[r.permutation(E)[:case["idle"]]] = 0.0
    return [int(m) * unit for m in r.multinomial(case["rows"] // unit, p / p.sum())]


def work(case):
    op = case["op"]
    nv = lambda rows, cols: rows * cols * 9 // 16 + 4 * rows  # noqa: E731  codes, block scales, row factors
    if op == "adapter":
        T, K, N, R = case["rows"], case["K"], case["N"], case["rank"]
        used = len({int(i) for i in _ids(case) if i >= 0})
        live = sum(int(i) >= 0 for i in _ids(case))
        return {"bytes": nv(T, K) + nv(N, K) + 2 * T * K + 2 * T * N + used * 2 * R * (K + N) + 4 * T,
                "flops": 2 * T * K * N + 2 * live * R * (K + N)}
    m = _splits(case)
    rows, live = sum(m), sum(v > 0 for v in m)
    if op == "gated_bwd":
        F = case["F"]
        return {"bytes": rows * F * 10 + 4 * rows + 8 * F * case["groups"], "flops": 20 * rows * F}
    K = case["K"]
    if op == "wgrad":
        N = case["N"]
        return {"bytes": rows * (N + K) * 9 // 16 + 4 * live * (N + K) + case["groups"] * N * K * (4 if case["fp32"] else 2),
                "flops": 2 * rows * N * K}
    N = case["N"] if op == "gemm" else 2 * case["F"]
    out = N if op == "gemm" else case["F"] * (3 if case["save"] else 1)
    return {"bytes": nv(rows, K) + live * nv(N, K) + 2 * rows * out, "flops": 2 * rows * K * N}


# ----------------------------------------------------------------- the inputs

def _tile(scale):
    """[rows, cols] block scales in tiles of 128 rows x 4 columns, 512 bytes
    each: byte (r % 32) * 16 + (r / 32) * 4 + c of its tile."""
    r, c = scale.shape
    return scale.view(r // 128, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(r, c)


def _cast(x, tiled):
    """NVFP4 with one factor a row of x [rows, cols] (fp32, on the GPU)."""
    rows, cols = x.shape
    amax = x.abs().amax(1) if cols else x.new_zeros(rows)
    enc = torch.where(amax > 0, 2688.0 / amax, torch.ones_like(amax))
    b = x.view(rows, cols // 16, 16)
    s8 = (b.abs().amax(2) / 6.0 * enc[:, None]).to(torch.float8_e4m3fn)
    f = s8.float()
    mul = torch.where(f > 0, enc[:, None] / f, torch.zeros_like(f))
    v = (b * mul[:, :, None]).view(rows, cols)
    code = torch.bucketize(v.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device),
                           out_int32=True).to(torch.uint8) + torch.signbit(v).to(torch.uint8) * 8
    s8 = s8.view(torch.uint8)
    return {"data": code[:, 0::2] + code[:, 1::2] * 16, "scale": _tile(s8) if tiled else s8, "s2": amax / 2688.0}


def _stack(parts, tiled):
    m = {k: torch.cat([p[k].reshape(-1) for p in parts]) for k in ("data", "scale", "s2")}
    m["scale_layout"] = int(tiled)
    return m


def _weights(E, N, K, g, tiled):
    """E matrices [N, K] of an initialised layer, cast along K."""
    step = max(1, (1 << 27) // (N * K))
    return _stack([_cast(torch.randn(min(step, E - e) * N, K, generator=g, device=DEV) * K ** -0.5, tiled)
                   for e in range(0, E, step)], tiled)


def _tokens(rows, K, g):
    """Activations: each row its own size, one row in 128 all zero (padding)."""
    x = torch.randn(rows, K, generator=g, device=DEV) * torch.exp2(
        torch.rand(rows, 1, generator=g, device=DEV) * 4 - 2)
    if rows > 1:
        x[torch.rand(rows, generator=g, device=DEV) < 1 / 128] = 0
    return x.to(torch.bfloat16)


def _cast_cols(x, m, tiled):
    """Each group's transpose, cast along its rows."""
    return _stack([_cast(p.float().t().contiguous(), tiled) for p in x.split(m)], tiled)


def _ids(case):
    """The adapter of each token: requests of uneven length lie one behind the
    other, one in eight of them without an adapter (-1)."""
    r = np.random.RandomState(case["routing"])
    n = case["requests"]
    cut = np.sort(r.choice(np.arange(1, case["rows"]), n - 1, replace=False)) if n > 1 else np.zeros(0, int)
    lens = np.diff(np.concatenate([[0], cut, [case["rows"]]])).astype(int)
    ids = r.permutation(max(n, case["adapters"]))[:n] % case["adapters"]
    ids[r.rand(n) < 0.125] = -1
    return np.repeat(ids, lens)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = case["op"], {"op": case["op"]}
    empty = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    if op == "adapter":
        T, K, N, R, L = case["rows"], case["K"], case["N"], case["rank"], case["adapters"]
        s["x_bf16"] = _tokens(T, K, g)
        s["x"] = _stack([_cast(s["x_bf16"].float(), case["tiled"])], case["tiled"])
        s["w"] = _weights(1, N, K, g, case["tiled"])
        s["a"] = (torch.randn(L, R, K, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
        s["b"] = (torch.randn(L, N, R, generator=g, device=DEV) * R ** -0.5).to(torch.bfloat16)
        s["factor"] = torch.rand(L, generator=g, device=DEV) * 2 + 0.25
        s["ids"] = torch.from_numpy(_ids(case).astype(np.int32)).to(DEV)
        s["y"] = empty(T, N)
        s["workspace"] = empty(T, R, dtype=torch.float32)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    m = s["m"] = _splits(case)
    rows, E = sum(m), case["groups"]
    if op == "gated_bwd":
        F = case["F"]
        s["dh"] = (_tokens(rows, F, g) * 0.01).to(torch.bfloat16)
        s["gate_up"] = _tokens(rows, 2 * F, g)
        s["d_gate_up"] = empty(rows, 2 * F)
        s["row_amax"], s["col_amax"] = empty(rows, dtype=torch.float32), empty(E * 2 * F, dtype=torch.float32)
        return s
    K = case["K"]
    x = _tokens(rows, K, g)
    if op == "wgrad":
        N = case["N"]
        s["x"] = _cast_cols(x, m, case["tiled"])
        s["dy"] = _cast_cols(_tokens(rows, N, g), m, case["tiled"])
        s["dw"] = empty(E, N, K, dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        return s
    s["x"] = _stack([_cast(x.float(), case["tiled"])], case["tiled"])
    if op == "gemm":
        s["w"] = _weights(E, case["N"], K, g, case["tiled"])
        s["y"] = empty(rows, case["N"])
    else:
        s["w"] = _weights(E, 2 * case["F"], K, g, case["tiled"])
        s["h"] = empty(rows, case["F"])
        s["gate_up"] = empty(rows, 2 * case["F"]) if case["save"] else None
    return s


# ------------------------------------------------------------- the plain form

def _values(data, scale, s2, tiled):
    """fp32 values [rows, cols] of one NVFP4 matrix with rows = len(s2)."""
    rows = s2.numel()
    pair = torch.tensor([[E2M1[n & 7] * (-1 if n & 8 else 1) for n in (b & 15, b >> 4)] for b in range(256)], device=DEV)
    v = pair.index_select(0, data.reshape(-1).int()).view(rows, -1, 16)
    s = scale.view(rows, -1)
    if tiled:
        s = s.view(rows // 128, -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rows, -1)
    return (v * s.view(torch.float8_e4m3fn).float()[:, :, None]).view(rows, -1) * s2[:, None]


def _products(x, m, w):
    """X_g W_g^T, one group at a time."""
    K = 2 * x["data"].numel() // x["s2"].numel()
    n = w["s2"].numel() // len(m)
    parts = zip(x["data"].split([r * K // 2 for r in m]), x["scale"].split([r * K // 16 for r in m]), x["s2"].split(m),
                w["data"].split(n * K // 2), w["scale"].split(n * K // 16), w["s2"].split(n))
    return torch.cat([_values(a, b, c, x["scale_layout"]) @ _values(d, e, f, w["scale_layout"]).t()
                      for a, b, c, d, e, f in parts if c.numel()])


def _plain(s):
    op = s["op"]
    if op == "gemm":
        return _products(s["x"], s["m"], s["w"]).to(s["y"].dtype)
    if op == "gated":
        p = _products(s["x"], s["m"], s["w"])
        gate, up = p.chunk(2, 1)
        h = (gate * (1 / (1 + torch.exp(-gate))) * up).to(torch.bfloat16)
        return h if s["gate_up"] is None else (h, p.to(torch.bfloat16))
    if op == "gated_bwd":
        dh, (gate, up) = s["dh"].float(), s["gate_up"].float().chunk(2, 1)
        sig = 1 / (1 + torch.exp(-gate))
        d = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1).to(torch.bfloat16)
        a = d.abs()
        cols = [p.amax(0) if p.shape[0] else p.new_zeros(p.shape[1]) for p in a.split(s["m"])]
        return d, a.amax(1), torch.cat(cols)
    if op == "wgrad":
        E, N, K = s["dw"].shape
        part = lambda q, n: zip(q["data"].split([n * r // 2 for r in s["m"]]), q["scale"].split([n * r // 16 for r in s["m"]]),  # noqa: E731
                                q["s2"].split(n))
        val = lambda d, c, f: _values(d, c, f, s["x"]["scale_layout"]) if d.numel() else d.new_zeros(f.numel(), 0).float()  # noqa: E731
        return torch.stack([(val(*p) @ val(*q).t()).to(s["dw"].dtype) for p, q in zip(part(s["dy"], N), part(s["x"], K))])
    x = s["x_bf16"].float()
    L, R, K = s["a"].shape
    y = _products(s["x"], [x.shape[0]], s["w"])
    # every token against every adapter's A, its own kept, then spread over its own B
    live = s["ids"][:, None] == torch.arange(L, device=DEV, dtype=torch.int32)[None, :]
    u = (x @ s["a"].float().view(L * R, K).t()).view(-1, L, R) * (live * s["factor"])[:, :, None]
    return (y + u.view(-1, L * R) @ s["b"].float().permute(0, 2, 1).reshape(L * R, -1)).to(s["y"].dtype)


def run(s):
    if not own:
        return _plain(s)
    from nvfp4_row_scaled_b200 import abi
    op = s["op"]
    if op == "gemm":
        abi.nvfp4_group_gemm(s["x"], s["m"], s["w"], s["y"])
        return s["y"]
    if op == "gated":
        abi.nvfp4_group_gated_gemm(s["x"], s["m"], s["w"], s["h"], gate_up=s["gate_up"])
        return s["h"] if s["gate_up"] is None else (s["h"], s["gate_up"])
    if op == "gated_bwd":
        abi.nvfp4_group_gated_backward(s["dh"], s["gate_up"], s["m"], s["d_gate_up"], s["row_amax"], s["col_amax"])
        # an amax is a bf16 value held in fp32: its upper half is that value
        return s["d_gate_up"], s["row_amax"].view(torch.bfloat16)[1::2], s["col_amax"].view(torch.bfloat16)[1::2]
    if op == "wgrad":
        abi.nvfp4_group_wgrad(s["dy"], s["x"], s["m"], s["dw"])
        return s["dw"]
    abi.nvfp4_adapter_gemm(s["x_bf16"], s["x"], s["w"], s["a"], s["b"], s["factor"], s["ids"], s["y"], s["workspace"],
                           s["status"])
    return s["y"]


# ------------------------------------------------------------- 64-bit results

def _exact_matrix(data, scale, s2, rows, cols, tiled):
    """fp64 [rows, cols], decoded from the bits of each code and scale."""
    d = data.reshape(rows, cols // 2)
    code = torch.empty(rows, cols, dtype=torch.uint8, device=d.device)
    code[:, 0::2] = d & 15
    code[:, 1::2] = d >> 4
    e, f = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e == 0, f * 0.5, (1 + f * 0.5) * torch.exp2(e.double() - 1))
    v = torch.where(code >= 8, -v, v)
    r = torch.arange(rows, device=d.device)[:, None]
    c = torch.arange(cols // 16, device=d.device)[None, :]
    at = r * (cols // 16) + c
    if tiled:
        at = ((r // 128) * (cols // 64) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    b = scale.reshape(-1)[at]
    e, f = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e.double() - 7))
    return (v.view(rows, -1, 16) * sc[:, :, None]).view(rows, cols) * s2.double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated_bwd":
        dh, gate, up = s["dh"].double(), *s["gate_up"].double().chunk(2, 1)
        sig = torch.sigmoid(gate)
        d = torch.cat([dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig], 1)
        col = torch.zeros(case["groups"], d.shape[1], dtype=torch.float64, device=d.device)
        o = 0
        for g, n in enumerate(s["m"]):
            if n:
                col[g] = d[o:o + n].abs().max(0).values
            o += n
        return d, d.abs().max(1).values, col.view(-1)
    if op == "wgrad":
        N, K, t, out, o = case["N"], case["K"], case["tiled"], [], 0
        for g, n in enumerate(s["m"]):
            pair = []
            for q, w in ((s["dy"], N), (s["x"], K)):
                pair.append(_exact_matrix(q["data"][w * o // 2:w * (o + n) // 2], q["scale"][w * o // 16:w * (o + n) // 16],
                                          q["s2"][g * w:(g + 1) * w], w, n, t))
            out.append(torch.matmul(pair[0], pair[1].t()))
            o += n
        return torch.stack(out)
    K, t = case["K"], case["tiled"]
    m = s["m"] if op != "adapter" else [case["rows"]]
    N = 2 * case["F"] if op == "gated" else case["N"]
    x, w = s["x"], s["w"]
    p = torch.empty(sum(m), N, dtype=torch.float64, device=DEV)
    o = 0
    for g, n in enumerate(m):
        if n:
            a = _exact_matrix(x["data"][o * K // 2:(o + n) * K // 2], x["scale"][o * K // 16:(o + n) * K // 16],
                              x["s2"][o:o + n], n, K, t)
            b = _exact_matrix(w["data"][g * N * K // 2:(g + 1) * N * K // 2], w["scale"][g * N * K // 16:(g + 1) * N * K // 16],
                              w["s2"][g * N:(g + 1) * N], N, K, t)
            torch.matmul(a, b.t(), out=p[o:o + n])
        o += n
    if op == "gemm":
        return p
    if op == "gated":
        F = case["F"]
        h = p[:, :F] * torch.sigmoid(p[:, :F]) * p[:, F:]
        return (h, p) if case["save"] else h
    ids = _ids(case)
    for a in sorted(set(int(i) for i in ids if i >= 0)):
        at = torch.from_numpy(np.nonzero(ids == a)[0]).to(DEV)
        u = s["x_bf16"][at].double() @ s["a"][a].double().t()
        p[at] += s["factor"][a].double() * (u @ s["b"][a].double().t())
    return p
