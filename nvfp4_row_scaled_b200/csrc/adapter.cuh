// adapter.cuh -- the first half of low-rank adapters beside a shared
// projection: u[t][r] = factor[a] sum_k x[t][k] A_a[r][k], a = id[t].
//
// The second half, sum_r u[t][r] B_a[n][r], is added in the epilogue of the
// shared projection (group_gemm.cuh, kGemmAdapter), so the projection's output
// is written once.
//
// Bound by memory: x is read once and each adapter in use once a token block;
// 2 R flop a byte of x at most. bf16 mma.sync tiles (16 tokens x 8 ranks x 16
// of k): with R <= 64 columns the work is a fraction of the time of the loads,
// and the fragments come straight from global memory, with no staging to wait
// for. The contraction order is free, so a lane's 16-byte load (8 consecutive
// k of one row) feeds two MMAs, its k pairs numbered alike on both sides.
//
// Work split. A token block of 16 kMT rows; its K is split over the 8 warps of a
// CTA and the `cn` CTAs of a cluster, the partial sums added in a fixed order
// (warps, then cluster ranks). cn is a function of K alone, so a token's result depends neither
// on timing nor on the rows and adapters of the call. The block's
// distinct adapters are dealt to `slots` CTAs: each multiplies the whole block by
// its adapters and keeps the rows that use them. A decode step (a different
// adapter on every row) runs its adapters side by side; a prompt has one
// adapter in most blocks and leaves the other slots empty.
// Measured: 8192 rows x 7168 at rank 32 in 54 us (x at 2.2 TB/s: 512 CTAs keep the SMs
// busy for 64% of it, and their warps wait for the row-wise loads; 1 to 3 CTAs a SM and 2 to 8
// steps unrolled are alike), 64 rows x 4096 with an adapter each at rank 16 in 8.5 us.
#pragma once

#include <cooperative_groups.h>

#include "bounds.cuh"
#include "routing.cuh"

namespace nvfp4rs {

namespace cg = cooperative_groups;

constexpr int kAdThreads = 256;
constexpr int kAdMaxRank = 64;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_u4(const uint4* p) {
  if (!NVFP4_LOAD_OK(p, 16)) return make_uint4(0u, 0u, 0u, 0u);
  return __ldg(p);
}

// kNT = rank / 8 column tiles. partial: dynamic shared [8 warps][16 kMT][8 kNT] floats.
template <int kMT, int kNT>
__global__ void __launch_bounds__(kAdThreads, 2)
adapter_shrink_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ A, const float* __restrict__ factor,
                      const int32_t* __restrict__ ids, float* __restrict__ u, int32_t* __restrict__ status,
                      int32_t rows, int32_t K, int32_t adapters, int32_t cn, int32_t slots) {
  constexpr int kTok = 16 * kMT, kR = 8 * kNT;
  __shared__ int32_t id[kTok];
  __shared__ int32_t distinct[kTok];
  __shared__ int32_t count;
  extern __shared__ float partial[];
  launch_dependents();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int slot = blockIdx.y;
  const int32_t t0 = static_cast<int32_t>(blockIdx.x / cn) * kTok;
  // the block's distinct adapters, in the order of their first tokens: one warp,
  // a lane for each token
  if (warp == 0) {
    int32_t a = lane < kTok && t0 + lane < rows ? gload(&ids[t0 + lane]) : -1;
    if (a >= adapters || a < -1) {
      if (slot == 0 && rank == 0) gstore(status, static_cast<int32_t>(NVFP4_ERR_ROUTING));
      a = -1;
    }
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, a);
    const bool first = a >= 0 && __ffs(same) - 1 == lane;
    const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, first);
    if (lane < kTok) id[lane] = a;
    if (first) distinct[__popc(firsts & ((1u << lane) - 1))] = a;
    if (lane == 0) count = __popc(firsts);
  }
  __syncthreads();
  const int n = count;
  // this warp's part of K, in steps of 32
  const int steps = (K + 31) / 32;
  const int parts = 8 * cn, part = rank * 8 + warp;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * part / parts);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / parts);
  const int gr = lane >> 2, kq = (lane & 3) * 8;
  // rows behind the last read the last one again: no branches around the loads
  const uint16_t* xr[kMT][2];
#pragma unroll
  for (int m = 0; m < kMT; m++)
#pragma unroll
    for (int h = 0; h < 2; h++) xr[m][h] = x + static_cast<int64_t>(min(t0 + 16 * m + 8 * h + gr, rows - 1)) * K + kq;
  // the loop count is the same in every CTA of the cluster (same tokens, same slot)
  for (int d = slot; d < n; d += slots) {
    const int32_t a = distinct[d];
    const uint16_t* Aa = A + static_cast<int64_t>(a) * kR * K;
    float acc[kMT][kNT][4];
#pragma unroll
    for (int m = 0; m < kMT; m++)
#pragma unroll
      for (int c = 0; c < kNT; c++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[m][c][e] = 0.0f;
    const uint16_t* ar = Aa + static_cast<int64_t>(gr) * K + kq;
    auto step = [&](int k, bool in) {
      uint4 xv[kMT][2], bv[kNT];
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int m = 0; m < kMT; m++)
#pragma unroll
        for (int h = 0; h < 2; h++) xv[m][h] = in ? ld_u4(reinterpret_cast<const uint4*>(xr[m][h] + k)) : zero;
#pragma unroll
      for (int c = 0; c < kNT; c++)
        bv[c] = in ? ld_u4(reinterpret_cast<const uint4*>(ar + static_cast<int64_t>(8 * c) * K + k)) : zero;
#pragma unroll
      for (int m = 0; m < kMT; m++)
#pragma unroll
        for (int c = 0; c < kNT; c++) {
          mma_bf16(acc[m][c], xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y, bv[c].x, bv[c].y);
          mma_bf16(acc[m][c], xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w, bv[c].z, bv[c].w);
        }
    };
    const int whole = min(s1, K / 32);
#pragma unroll 4
    for (int s = s0; s < whole; s++) step(32 * s, true);
    if (s1 > whole && s1 > s0) step(32 * (s1 - 1), 32 * (s1 - 1) + kq < K);  // the last half step of a K off the 32s
    float* mine = partial + warp * kTok * kR;
#pragma unroll
    for (int m = 0; m < kMT; m++)
#pragma unroll
      for (int c = 0; c < kNT; c++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          mine[(16 * m + gr + (e >> 1) * 8) * kR + 8 * c + (lane & 3) * 2 + (e & 1)] = acc[m][c][e];
    __syncthreads();
    for (int i = t; i < kTok * kR; i += kAdThreads) {
      float s = partial[i];
#pragma unroll
      for (int w = 1; w < 8; w++) s += partial[w * kTok * kR + i];
      partial[i] = s;
    }
    cluster.sync();
    if (rank == 0) {
      const float f = gload(&factor[a]);
      for (int i = t; i < kTok * kR; i += kAdThreads)
        if (id[i / kR] == a) {
          float s = partial[i];
          for (int q = 1; q < cn; q++) s += *cluster.map_shared_rank(&partial[i], q);
          gstore(&u[static_cast<int64_t>(t0) * kR + i], s * f);
        }
    }
    cluster.sync();  // the partial sums are free again
  }
}

}  // namespace nvfp4rs
