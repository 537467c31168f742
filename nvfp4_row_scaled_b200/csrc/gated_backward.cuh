// gated_backward.cuh -- gradient of the gated product, with the amax of its cast.
//
// For h = silu(g) u with the saved pre-activations (g, u) = gate_up[t][f],
// gate_up[t][F + f] and the incoming dh:
//   d_gate = dh u s (1 + g (1 - s)),   d_up = dh g s,   s = 1 / (1 + e^-g)
// in fp32 (gated_grad below has the form that keeps its range), rounded once to
// bf16 into d_gate_up [rows][2F]. That buffer is cast to NVFP4 next (both directions: the input gradient reads the rows, the
// weight gradient the columns), so the same pass also yields what the grouped
// amax of it would (TransformerEngine #3649, Description): the row amax and the
// per-group column amax of the ROUNDED values, bit for bit, which saves that
// step's read of the buffer (4 bytes of 14 a gradient pair).
//
// Bound by memory: 6 bytes in and 4 out for each element of h.
//
// Work split. A tile is 64 rows of the packed buffer, its 256-column chunks of
// F dealt round robin to a cluster of `cn` CTAs. Eight warps: four 16-row
// blocks (each inside one group) x two chunks at a time. A lane owns 8 columns
// and walks the 16 rows, 4 at a time with 12 16-byte loads in flight; its 16
// column maxima stay in registers over the rows, its 16 row maxima over the
// chunks. Column maxima meet in shared memory and leave with one unsigned
// atomic max a column (order-free, so deterministic); a tile that a group
// boundary crosses sends each block's maxima straight to its group. Row maxima
// meet in shared memory and, over the cluster, in CTA 0. Smaller tiles would
// need more atomics, larger ones leave a packed batch of a few thousand rows
// on too few SMs.
#pragma once

#include "codec.cuh"
#include "group_amax.cuh"
#include "post_scale.cuh"
#include "routing.cuh"

namespace nvfp4rs {

constexpr int kBwThreads = 256;
constexpr int kBwRows = 64;
constexpr int kBwChunk = 256;  // columns of F: 32 lanes x 8

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// In place, gate_up is the output: its loads are ordinary ones that keep their place before the
// stores of the same rows. Elsewhere they take the read-only path, which wants memory that
// nothing writes meanwhile and whose loads the compiler may move over the stores
// (80768 x 2048: 320 us, 350 with the ordered loads).
template <bool kInPlace>
__device__ __forceinline__ uint4 ld_gate_up(const uint4* p) {
  if (!kInPlace) return ld_stream(p);
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (!NVFP4_LOAD_OK(p, 16)) return v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// streaming: 322 us against 338 with plain stores at 80768 x 2048 (5.1 TB/s)
__device__ __forceinline__ void st_stream(uint4* p, uint4 v) {
  if (NVFP4_STORE_OK(p, 16)) __stcs(p, v);
}

// One element: (d_gate, d_up). With h = e^(-|g|/2), m = 1 for g >= 0 and h below, r = 1 / (1 + h^2):
// s = m^2 r and 1 - s = (g >= 0 ? h^2 : 1) r, with no cancellation, no divisor above 2 and
// no s below 2^-126 on its own: dh and u take a factor m each (either way round some products of
// huge and tiny factors leave fp32's range; here those with |dh| m or |u| m below 2^-126).
__device__ __forceinline__ float2 gated_grad(float dh, float g, float u) {
  const float h = half_exp(g), q = h * h, r = fast_rcp(1.0f + q);
  const bool pos = g >= 0.0f;
  const float m = pos ? 1.0f : h, d = dh * m, mr = m * r;
  return make_float2(d * (u * mr) * __fmaf_rn(g, (pos ? q : 1.0f) * r, 1.0f), d * (g * mr));
}

template <class Routing, bool kInPlace>
__global__ void __launch_bounds__(kBwThreads, 2)
gated_backward_kernel(const __grid_constant__ Routing routing, const uint4* __restrict__ dh, const uint4* gate_up,
                      uint4* out, int32_t F, int32_t cn,
                      float* __restrict__ row_amax, float* __restrict__ col_amax) {
  __shared__ RoutingSmem rs;
  __shared__ uint32_t rmax[kBwRows];
  extern __shared__ uint32_t cmax[];  // [chunks of this CTA][gate 256, up 256], then the group offsets
  launch_dependents();
  const int nch = (F + kBwChunk - 1) / kBwChunk;
  const int per = (nch + cn - 1) / cn;
  routing.load(rs, reinterpret_cast<int32_t*>(cmax + per * 2 * kBwChunk));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rb = warp & 3, hf = warp >> 2;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int32_t r0 = static_cast<int32_t>(blockIdx.x / cn) * kBwRows;
  const bool active = rs.ok && r0 < rs.total;
  const int valid = active ? min(kBwRows, rs.total - r0) : 0;  // a multiple of 16
  const bool block_ok = 16 * rb < valid;
  const int g_first = active ? group_of_row(rs, r0) : 0;
  const bool mixed = active && rs.off[g_first + 1] < r0 + valid;
  const int g_block = mixed && block_ok ? group_of_row(rs, r0 + 16 * rb) : g_first;
  if (t < kBwRows) rmax[t] = 0u;
  for (int c = t; c < per * 2 * kBwChunk; c += kBwThreads) cmax[c] = 0u;
  __syncthreads();

  if (block_ok) {
    const size_t p8 = static_cast<size_t>(F) >> 3;  // row pitch of dh in 16-byte units
    const size_t row = static_cast<size_t>(r0) + 16 * rb;
    uint32_t rm[16];
#pragma unroll
    for (int i = 0; i < 16; i++) rm[i] = 0u;
    for (int j = hf; j < per; j += 2) {
      const int c0 = (j * cn + rank) * kBwChunk + lane * 8;
      if (c0 < F) {
        const uint4* pd = dh + row * p8 + (c0 >> 3);
        const uint4* pg = gate_up + row * 2 * p8 + (c0 >> 3);
        uint4* po = out + row * 2 * p8 + (c0 >> 3);
        uint32_t cg4[4] = {0u, 0u, 0u, 0u}, cu4[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i0 = 0; i0 < 16; i0 += 4) {
          uint4 d[4], g[4], u[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            d[i] = ld_stream(pd + (i0 + i) * p8);
            g[i] = ld_gate_up<kInPlace>(pg + (i0 + i) * 2 * p8);
            u[i] = ld_gate_up<kInPlace>(pg + (i0 + i) * 2 * p8 + p8);
          }
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const uint32_t dw[4] = {d[i].x, d[i].y, d[i].z, d[i].w}, gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w},
                           uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
            uint32_t og[4], ou[4];
#pragma unroll
            for (int q = 0; q < 4; q++) {
              const float2 a = gated_grad(bf16_lo(dw[q]), bf16_lo(gw[q]), bf16_lo(uw[q]));
              const float2 b = gated_grad(bf16_hi(dw[q]), bf16_hi(gw[q]), bf16_hi(uw[q]));
              og[q] = bf16x2_rn(a.x, b.x);
              ou[q] = bf16x2_rn(a.y, b.y);
              cg4[q] = maxabs2(cg4[q], og[q]);
              cu4[q] = maxabs2(cu4[q], ou[q]);
              rm[i0 + i] = maxabs2(rm[i0 + i], maxabs2(og[q], ou[q]));
            }
            st_stream(po + (i0 + i) * 2 * p8, make_uint4(og[0], og[1], og[2], og[3]));
            st_stream(po + (i0 + i) * 2 * p8 + p8, make_uint4(ou[0], ou[1], ou[2], ou[3]));
          }
        }
        if (col_amax != nullptr) {
          if (mixed) {  // straight to this block's group (a mixed tile is rare)
            grid_dependency_wait();  // col_amax is zero
            float* cgp = col_amax + static_cast<size_t>(g_block) * 2 * F + c0;
#pragma unroll
            for (int q = 0; q < 4; q++) {
              red_max_u32(cgp + 2 * q, (cg4[q] & 0x7FFFu) << 16);
              red_max_u32(cgp + 2 * q + 1, cg4[q] & 0x7FFF0000u);
              red_max_u32(cgp + F + 2 * q, (cu4[q] & 0x7FFFu) << 16);
              red_max_u32(cgp + F + 2 * q + 1, cu4[q] & 0x7FFF0000u);
            }
          } else {
            uint32_t* cm = cmax + j * 2 * kBwChunk + lane * 8;
#pragma unroll
            for (int q = 0; q < 4; q++) {
              atomicMax(cm + 2 * q, (cg4[q] & 0x7FFFu) << 16);
              atomicMax(cm + 2 * q + 1, cg4[q] & 0x7FFF0000u);
              atomicMax(cm + kBwChunk + 2 * q, (cu4[q] & 0x7FFFu) << 16);
              atomicMax(cm + kBwChunk + 2 * q + 1, cu4[q] & 0x7FFF0000u);
            }
          }
        }
      }
    }
    if (row_amax != nullptr) {
#pragma unroll
      for (int i = 0; i < 16; i++) {
        const uint32_t m = max(rm[i] & 0x7FFFu, (rm[i] >> 16) & 0x7FFFu);
        const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, m);
        if (lane == 0) atomicMax(&rmax[16 * rb + i], w << 16);
      }
    }
  }
  __syncthreads();
  // col_amax is zero; waited for by every CTA, those without rows too: what follows on the stream
  // waits for this kernel and not for the zeroing before it
  if (col_amax != nullptr) grid_dependency_wait();
  if (active && !mixed && col_amax != nullptr) {
    float* dst = col_amax + static_cast<size_t>(g_first) * 2 * F;
    for (int c = t; c < per * 2 * kBwChunk; c += kBwThreads) {
      const int col = ((c / (2 * kBwChunk)) * cn + rank) * kBwChunk + (c & (kBwChunk - 1));
      if (col < F) red_max_u32(dst + ((c & kBwChunk) ? F : 0) + col, cmax[c]);
    }
  }
  // every CTA of the cluster reaches both barriers, active or not
  cluster.sync();
  if (rank == 0 && row_amax != nullptr && t < valid) {
    uint32_t m = rmax[t];
    for (int q = 1; q < cn; q++) m = max(m, *cluster.map_shared_rank(&rmax[t], q));
    gstore(&row_amax[r0 + t], __uint_as_float(m));
  }
  cluster.sync();
}

}  // namespace nvfp4rs
