// group_gemm.cuh -- products of grouped row-scaled NVFP4 matrices on the
// block-scaled tensor cores.
//
// What the casts of this library are made for (TransformerEngine #2931,
// "Implement per-token NVFP4 fprop recipe", sequence diagram: a GEMM over the
// row-scaled operands whose output is multiplied back by the row factors;
// #3324, the row-scaled backward of the grouped linear layer). One kernel
// body serves
//   kGemmPlain    y[t][n]  = sx[t] sw[n] sum_k x[t][k] w_g[n][k]      (t in group g)
//   kGemmGated    h[t][f]  = silu(p[t][f]) * p[t][F + f],  p as above, N = 2F
//   kGemmWgrad    dw_g[n][k] = sdy[n] sx[k] sum_t dy[t][n] x[t][k]    (t in group g)
//   kGemmAdapter  kGemmPlain + sum_r u[t][r] b_a[n][r],  a = id[t]
// where every x, w, dy is e2m1 * e4m3 (a code and the scale of its 16-element
// block) and s.. the fp32 row factor of the cast.
//
// The mathematics on the hardware. A tcgen05.mma of kind mxf4nvf4 multiplies
// 64 codes of each row, applies both operands' E4M3 scales per 16 codes and
// accumulates in fp32 in tensor memory; the row factors are constant along
// the contraction, so they are applied once, in fp32, when the accumulator is
// read: fl(fl(acc * s_J) * s_I). The result is rounded once to the output type.
//
// Orientation. Accumulator LANES (128, the M side of the instruction) are
// rows of operand I -- weights, or for wgrad the columns of x -- and COLUMNS
// (N side, any multiple of 16 up to 256) rows of operand J -- tokens, or the
// columns of dy. The token side is the one whose length varies, from one row
// to thousands, and the N side is the one that can be cut to 16: a group of
// one token costs 16 columns, not 128 lanes, while a decode step streams its
// weights 128 rows at a time. out[J row][I row] is then row-major with the 32
// lanes of a warp on 32 neighbouring elements.
//
// Work split. A persistent CTA per SM walks every gridDim-th tile (128 I rows
// x `jt` J rows of one group, I tiles innermost so that concurrent CTAs share
// the token tile and the group's weights in L2). Large problems run it on pairs
// of CTAs (kPair): 256 I rows, 128 to a CTA, x up to 256 J rows of which each CTA
// loads half, in one MMA over both SMs' tensor cores. Why pairs: an SM reads 64 bytes
// a cycle from L2, and a 256-element k block of a 128 x 256 tile is 512 cycles of MMA and
// 54 KB (864 cycles) to one CTA, 38 KB (608) to each of a pair (gated: 46 KB, 736). A block
// takes about 790 cycles at 8192 x 8192 x 8192 and 829 in a gated call of 80768 rows x 7168, under the
// power cap's 1.40 and 1.14 GHz; at K = 2048, where a tile has 8 blocks and its stores take as
// long, 970 to 1360. Five roles, joined by mbarriers:
//   warp 0      data of each 256-element k block by TMA (128-byte swizzle) and
//               tiled block scales by bulk copies
//   warp 1      tensor memory, scale copies shared -> tensor memory, MMAs (in
//               a pair the first CTA's; the second's passes on that its stage
//               has been filled)
//   warps 4-7   what TMA cannot address, a stage to a warp: row-major block
//               scales (16 bytes a row and k block, read ahead into registers
//               and written as the 128x4 tiles the MMA wants) and, with kTma =
//               false, the codes themselves (row strides that are not
//               multiples of 16 bytes; wgrad's per-group strides)
//   warps 8-15  epilogue: two warps for each 32-lane quarter, alternate
//               32-column chunks
// Tensor memory holds two 256-column accumulators at columns 0 and 192 that
// share 64 columns, and 48 columns of scales behind them: the next tile's
// MMAs start once the shared columns of this one have been read, which the
// epilogue does first.
//
// Measured (30 calls in a row): 8192 x 8192 x 8192 in 216 us (5.1 PFLOP/s; in a loop of seconds 249
// us, 4.4), 288 with row-major scales; 128 experts of a few tokens in 58 us, 4.8 TB/s of
// all bytes; 16 fp32 weight gradients of 2048 x 4096 in 107 us, 5.0 TB/s of stores.
//
// Every wait is bounded. After a give-up the roles leave their loops, wait
// (bounded) for what is in flight, and the status is reported where the call
// has a status word.
#pragma once

#include <cuda.h>

#include "group_cast.cuh"
#include "adapter.cuh"
#include "post_scale.cuh"
#include "routing.cuh"

namespace nvfp4rs {

enum GemmMode : int { kGemmPlain = 0, kGemmGated = 1, kGemmWgrad = 2, kGemmAdapter = 3 };

constexpr int kGThreads = 512;       // warpgroups: TMA and MMA warps (two idle), loaders, 2 of epilogue
constexpr int kGLoadWarp = 4;
constexpr int kGEpiWarp = 8;
constexpr int kGEpiWarps = 8;
// registers a thread: 128 at launch; the first warpgroup gives 64 of them up and
// the two of the epilogue take 32 each (the loaders keep theirs)
constexpr int kGRegsLaunch = 65536 / kGThreads, kGRegsIssue = 64, kGRegsEpi = 160;
static_assert(kGRegsIssue <= kGRegsLaunch && kGRegsEpi >= kGRegsLaunch &&
                  kGRegsIssue + kGRegsLaunch + 2 * kGRegsEpi <= 4 * kGRegsLaunch,
              "register split");
constexpr int kGI = 128;             // I rows (accumulator lanes) of a CTA's tile
constexpr int kGK = 256;             // contraction elements of a stage: 128 bytes a row
constexpr int kGBigJ = 128;          // J rows of a TMA box ...
constexpr int kGBoxJ = 32;           // ... and of one in a tile's rest
constexpr int kGIBytes = kGI * 128;
constexpr int kGScaleTile = 512;     // 128 rows x 4 scales
constexpr int kGSfBytes = 3 * 4 * kGScaleTile;  // I and two blocks of 128 J rows (gated: gate, up, J), 4 k steps
constexpr int kGAcc1 = 192;          // first column of the second accumulator
constexpr int kGSfCol = 448;         // first scale column

// A stage: I codes (gated: gate, then up), the CTA's J codes, scales.
template <bool kGated>
struct GemmStage {
  static constexpr int kJRows = kGated ? 64 : 128;  // J rows a CTA holds; a pair's tile has twice as many
  static constexpr int kIData = kGated ? 2 * kGIBytes : kGIBytes;
  static constexpr int kData = kIData + kJRows * 128;
  static constexpr int kISf = (kGated ? 2 : 1) * 4 * kGScaleTile;
  static constexpr int kBytes = kData + kGSfBytes;
  static constexpr int kStages = kGated ? 4 : 5;
  static_assert(kStages >= 4, "four loader warps, a stage each");
};

struct GemmOperand {
  const uint8_t* data;
  const uint8_t* scale;
  const float* s2;
  int32_t tiled;  // block scales in 128x4 tiles
};

struct GemmArgs {
  GemmOperand i, j;
  int32_t ni;        // output columns: I rows of a group (gated: of each half)
  int32_t nj;        // wgrad: J rows of a group
  int32_t K;         // contraction (wgrad: the group's rows instead)
  int32_t j_whole;   // J rows whose row-major scales lie in whole aligned words: all, or all but the last one to three
  int32_t jt, jt_log;       // J rows of a tile: a power of two, 16 to 256; its logarithm
  uint32_t it, it_magic;    // I tiles of a group; floor(2^32 / it), 2^32 - 1 for it = 1
  int32_t jbulk;     // nonzero: J scales by bulk copies (tiled, and J tiles of whole 128-row blocks)
  int32_t loaders;   // nonzero: warps 4-7 take part
  int32_t producer;  // nonzero: warp 0 takes part
  int32_t out_f32;
  void* out;         // [J rows][ni]
  uint16_t* pre;     // gated: bf16 [rows][2 ni] or null
  // adapters
  const float* u;          // [rows][rank], already scaled
  const int32_t* ids;      // [rows]
  const uint16_t* b;       // bf16 [adapters][ni][rank]
  int32_t rank, adapters;
  int32_t* status;         // or null
};

template <bool kGated>
struct GemmSmem {
  using Stage = GemmStage<kGated>;
  uint8_t stage[Stage::kStages][Stage::kBytes];
  uint32_t turn[kGEpiWarps][16][32];     // an epilogue warp's chunk, row pairs x features
  float sj[kGEpiWarps][32];              // the J factors of an epilogue warp's chunk
  uint64_t full[Stage::kStages];
  uint64_t peer_full[Stage::kStages];    // pair, first CTA: the second's stage is full
  uint64_t empty[Stage::kStages];
  uint64_t acc_full;
  uint64_t acc_free;                     // pair: the first CTA's, for both epilogues
  uint64_t drain;
  uint32_t tmem;
  uint32_t gave_up;
  RoutingSmem routing;
};

template <bool kGated>
constexpr size_t gemm_smem_bytes(int E) {
  return ((sizeof(GemmSmem<kGated>) + 15) & ~size_t{15}) + sizeof(int32_t) * (static_cast<size_t>(E) + 1);
}

// ------------------------------------------------------------------ tcgen05

// Shared-memory matrix descriptor, K-major, 128-byte swizzle: rows of 128
// bytes, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t mma_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (uint64_t{1} << 16) | (uint64_t{1024 >> 4} << 32) |
         (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
// Descriptor of a 512-byte scale tile (32 rows of 16 bytes, no swizzle): 8-row
// groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (uint64_t{1} << 16) | (uint64_t{128 >> 4} << 32) |
         (uint64_t{1} << 46);
}
// Instruction descriptor of kind mxf4nvf4: E2M1 x E2M1, UE4M3 scales, M = 128
// (256 in a pair), N = n (a multiple of 16), both operands K-major.
template <bool kPair>
__device__ __forceinline__ uint32_t mma_idesc(int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((kPair ? 2u : 1u) << 27);
}

template <bool kPair>
__device__ __forceinline__ void mma_nvf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, bool accumulate) {
  if (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// a 512-byte scale tile to four columns of every lane quarter (a pair: of both
// CTAs, each from its own shared memory)
template <bool kPair>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  if (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// an arrival on `bar` (a pair: on both CTAs' one) once the MMAs issued so far are done
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if (kPair)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_addr(bar)),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
  if (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void tmem_dealloc(uint32_t tmem) {
  if (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}
// Arrival on the same barrier of the pair's first CTA. What it orders is not
// this thread's own writes but the tensor core's and TMA's (already complete:
// the thread has waited for them), so the default release is enough; one of
// cluster scope flushes the thread's memory path and halved the product's rate.
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_addr(bar)));
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive accumulator columns of the warp's 32 lanes (not yet waited for)
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
// the registers pass through it, so that no use of them is scheduled before it
__device__ __forceinline__ void tmem_load_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}

// --------------------------------------------------------------- cp.async

// 4, 8 or 16 bytes global -> shared of which the first `valid` are read and
// the rest zeroed; `src` is a real address even when valid == 0
template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const uint8_t* src, int valid) {
  if (!NVFP4_LOAD_OK(src, valid > 0 ? valid : 0)) valid = 0;
  if (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(valid)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// --------------------------------------------------------------- tile walk

struct GemmTile {
  int32_t kc;       // contraction length
  int32_t i0, j0;   // first I row of this CTA and first J row, inside the group's matrices
  int32_t iv, jv;   // I rows of this CTA (0..128) and J rows of the tile (<= jt)
  int64_t irow;     // first I row: in the stacked matrix, or (wgrad) in the s2 vector
  int64_t jrow;     // first J row, likewise; also the output row
  int64_t goff;     // wgrad: the group's first routed row
};

// The tiles of a CTA, one after the other: index first(), first() + step(), ...
// over the groups' tiles in order. Every role walks them for itself, so a step
// costs no integer division: jt is a power of two, and the I tiles of a group are
// divided out with a reciprocal (a.it_magic = floor(2^32 / it), one short at most).
template <int kMode, bool kPair>
struct GemmWalk {
  static constexpr int kI = kPair ? 2 * kGI : kGI;  // I rows of a tile
  const RoutingSmem& rs;
  const GemmArgs& a;
  int32_t g = -1;          // group of the last tile found,
  int32_t row = 0, m = 0;  // its first routed row and its rows
  uint32_t t;              // next tile index
  uint32_t before = 0, end = 0;  // tile indices of group g
  __device__ __forceinline__ GemmWalk(const RoutingSmem& r, const GemmArgs& x) : rs(r), a(x) {
    t = kPair ? blockIdx.x >> 1 : blockIdx.x;  // both CTAs of a pair take the same
  }

  __device__ __forceinline__ bool next(GemmTile& tile) {
    while (t >= end) {
      if (++g >= rs.E) return false;
      row = rs.off[g];
      m = rs.off[g + 1] - row;
      before = end;
      end += static_cast<uint32_t>(((kMode == kGemmWgrad ? a.nj : m) + a.jt - 1) >> a.jt_log) * a.it;
    }
    const uint32_t local = t - before;
    t += kPair ? gridDim.x >> 1 : gridDim.x;
    uint32_t jb = __umulhi(local, a.it_magic);
    uint32_t ib = local - jb * a.it;
    if (ib >= a.it) {
      jb++;
      ib -= a.it;
    }
    const int32_t jn = kMode == kGemmWgrad ? a.nj : m;
    tile.kc = kMode == kGemmWgrad ? m : a.K;
    tile.i0 = static_cast<int32_t>(ib) * kI;
    tile.iv = min(kGI, a.ni - tile.i0);
    if (kPair && (blockIdx.x & 1)) {
      // the second CTA's rows; with none left it works on the first's again and stores nothing
      const int32_t left = a.ni - tile.i0 - kGI;
      tile.iv = max(0, min(kGI, left));
      if (left > 0) tile.i0 += kGI;
    }
    tile.j0 = static_cast<int32_t>(jb << a.jt_log);
    tile.jv = min(a.jt, jn - tile.j0);
    tile.goff = row;
    const int32_t in = kMode == kGemmGated ? 2 * a.ni : a.ni;
    tile.irow = static_cast<int64_t>(g) * in + tile.i0;
    tile.jrow = (kMode == kGemmWgrad ? static_cast<int64_t>(g) * a.nj : row) + tile.j0;
    return true;
  }
};

// Position in the ring of stages.
template <int kStages>
struct GemmRing {
  uint32_t s = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == kStages) {
      s = 0;
      phase ^= 1;
    }
  }
};

// The k blocks of a CTA's tiles, one after the other.
template <int kMode, bool kPair>
struct GemmBlocks {
  GemmWalk<kMode, kPair> walk;
  GemmTile t;
  int32_t kb, nkb;
  bool more;
  __device__ __forceinline__ GemmBlocks(const RoutingSmem& r, const GemmArgs& x) : walk(r, x), kb(0) { tile(); }
  __device__ __forceinline__ void tile() {
    while ((more = walk.next(t))) {
      nkb = (t.kc + kGK - 1) / kGK;
      if (nkb > 0) return;
    }
  }
  __device__ __forceinline__ void next() {
    if (++kb < nkb) return;
    kb = 0;
    tile();
  }
};

// ------------------------------------------------------------- loader roles

// A k block's codes of `rows` rows (`valid` of them real, the rest zeros; rows a
// multiple of 8), 128 bytes a row, kCopy bytes a copy, into the swizzled stage, by
// one warp. Eight rows at a time: a lane's places in the swizzle pattern and its
// distance to the rows' ends stay the same, so a copy costs three instructions.
template <int kCopy>
__device__ __forceinline__ void load_codes(uint32_t dst, const uint8_t* data, int64_t row_bytes, int rows, int valid,
                                           int32_t kbyte, int lane) {
  constexpr int kPer = 128 / kCopy, kRows = 32 / kPer, kSteps = 8 / kRows;
  const int r0 = lane / kPer, o = (lane % kPer) * kCopy;
  const int64_t left = row_bytes - kbyte - o;
  const int n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(kCopy), left)));
  const uint8_t* src = n > 0 ? data + r0 * row_bytes + kbyte + o : data;
  const int64_t step = n > 0 ? kRows * row_bytes : 0;
  uint32_t d[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; i++) {
    const int r = r0 + i * kRows;
    d[i] = dst + r * 128 + ((((o >> 4) ^ r) << 4) | (o & 15));
  }
#pragma unroll 2
  for (int rb = 0; rb < rows; rb += 8) {
#pragma unroll
    for (int i = 0; i < kSteps; i++) {
      const bool in = rb + r0 + i * kRows < valid;
      cp_async<kCopy>(d[i] + rb * 128, in ? src : data, in ? n : 0);
      src += step;
    }
  }
}

// How a thread reads the 16 scales of a row and k block: one load where the rows
// are 16-byte aligned (a warp's 32 rows are 32 lines, and every load instruction
// pays for each), four words where they are 4-byte aligned, the five words
// around them where rows start at any byte, four words 512 bytes apart out of
// 128x4 tiles.
enum ScaleRead : int { kRead16 = 0, kReadWords = 1, kReadBytes = 2, kReadTiled = 3 };

// `left`: scales from p to the row's end. What is read raw is put together by
// scale_words() later, so that a read is not waited for here. Every aligned word that is
// read lies in the matrix: the rows that own a byte of a word that the matrix ends inside
// (from row a.j_whole on) are read byte by byte, by patch_scales(). A check of the end in
// each read took 5003 ragged rows of 4096 from 108 to 121 us.
__device__ __forceinline__ void read_scales(const uint8_t* p, int how, int32_t left, uint32_t (&w)[5]) {
#pragma unroll
  for (int k = 0; k < 5; k++) w[k] = 0u;
  if (p == nullptr) return;
  if (how == kRead16) {
    const uint4 v = gload(reinterpret_cast<const uint4*>(p));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if (how == kReadBytes) {
    const int b = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3);
#pragma unroll
    for (int k = 0; k < 5; k++)
      if (4 * k < min(left, 16) + b) w[k] = gload(reinterpret_cast<const uint32_t*>(p - b) + k);
  } else {
    const int step = how == kReadTiled ? kGScaleTile / 4 : 1;
#pragma unroll
    for (int k = 0; k < 4; k++)
      if (4 * k < left) w[k] = gload(reinterpret_cast<const uint32_t*>(p) + k * step);
  }
}
// shift: bits from the first word's start to the first scale (kReadBytes)
__device__ __forceinline__ void scale_words(uint32_t shift, int32_t left, uint32_t (&w)[5]) {
#pragma unroll
  for (int k = 0; k < 4; k++) {
    w[k] = __funnelshift_r(w[k], w[k + 1], shift);
    const int n = left - 4 * k;
    if (n < 4) w[k] = n <= 0 ? 0u : w[k] & (0xFFFFFFFFu >> (8 * (4 - n)));
  }
}
// The 16 scales each of rows lane, lane + 32, lane + 64 and lane + 96 of a 128-row
// block into 128x4 tiles: scale (r, 4 k + b) at tile k, byte (r % 32) * 16 + (r / 32) * 4 + b.
__device__ __forceinline__ void store_scales(uint8_t* dst, int lane, const uint32_t (&w)[4][5]) {
#pragma unroll
  for (int k = 0; k < 4; k++)
    *reinterpret_cast<uint4*>(dst + k * kGScaleTile + lane * 16) = make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
}

// Rows j0 .. j1 - 1 of a tile's J scales, a byte a lane (`src`: the first one's scales of the
// k block, `cols` to the next row's, `left` to the row's end), over the zeros that store_scales() put there.
__device__ __forceinline__ void patch_scales(uint8_t* dst, const uint8_t* src, int32_t cols, int32_t left, int j0, int j1,
                                             int lane) {
  __syncwarp();
  if (lane >= min(left, 16)) return;
  for (int j = j0; j < j1; j++, src += cols)
    dst[((j >> 7) * 4 + (lane >> 2)) * kGScaleTile + (j & 31) * 16 + ((j & 127) >> 5) * 4 + (lane & 3)] = gload(src + lane);
}

__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t pair2(uint32_t lo, uint32_t hi) { return static_cast<uint64_t>(hi) << 32 | lo; }
__device__ __forceinline__ uint32_t bf16_pair(uint64_t v) { return bf16x2_rn(lo2(v), hi2(v)); }
// silu(g) u of a pair, g u / (1 + e^-g), as (g m / (1 + h^2)) (u m) with h = e^(-|g|/2) and m = 1 for
// g >= 0, h below. The divisor is at most 2 (a fast quotient by e^-g is 0 from
// 2^126 on), and h is a normal number down to g = -174.6, so that a large u still meets a
// silu(g) far below 2^-126; below that the product, under 2^-116, is 0. Hardware exponential and
// reciprocal: within a few parts in 2^23, plus |g| 2^-23 for the exponent's rounded argument.
__device__ __forceinline__ uint64_t silu_times2(uint64_t g, uint64_t u) {
  const float t0 = half_exp(lo2(g)), t1 = half_exp(hi2(g));
  const uint64_t h = pack2(t0, t1), m = pack2(lo2(g) >= 0.0f ? 1.0f : t0, hi2(g) >= 0.0f ? 1.0f : t1);
  const uint64_t d = fma2x(h, h, pack2(1.0f, 1.0f));
  return mul2x(mul2x(mul2x(g, m), pack2(fast_rcp(lo2(d)), fast_rcp(hi2(d)))), mul2x(u, m));
}

// 32 rows x 32 features of a warp, lane = feature, y[i] = rows 2i and 2i + 1 as
// bf16 pairs: turned in shared memory, stored as 16 bytes (8 features) a lane, so that
// an instruction writes 64 contiguous bytes of each of 8 rows. Stored one
// element a lane (2 bytes, 32 instructions and their predicates) a 128 x 256
// tile took 15 k cycles, turned by lane exchanges 8 k.
__device__ __forceinline__ void store_bf16(const uint32_t (&y)[16], uint32_t (&turn)[16][32], uint16_t* out,
                                           int64_t pitch, int rows, int features, int lane) {
  __syncwarp();  // the last chunk has been read
#pragma unroll
  for (int i = 0; i < 16; i++) turn[i][lane] = y[i];
  __syncwarp();
  const int f = (lane & 3) * 8;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int i = 8 * h + (lane >> 2);
    // odd row pairs read their second half first: two row pairs would share banks
    const bool odd = i & 1;
    const uint4 a = *reinterpret_cast<const uint4*>(&turn[i][f + (odd ? 4 : 0)]);
    const uint4 b = *reinterpret_cast<const uint4*>(&turn[i][f + (odd ? 0 : 4)]);
    const uint4 p = odd ? b : a, q = odd ? a : b;
    const uint4 lo = make_uint4(__byte_perm(p.x, p.y, 0x5410), __byte_perm(p.z, p.w, 0x5410),
                                __byte_perm(q.x, q.y, 0x5410), __byte_perm(q.z, q.w, 0x5410));
    const uint4 hi = make_uint4(__byte_perm(p.x, p.y, 0x7632), __byte_perm(p.z, p.w, 0x7632),
                                __byte_perm(q.x, q.y, 0x7632), __byte_perm(q.z, q.w, 0x7632));
    if (f < features) {
      uint16_t* o = out + 2 * i * pitch + f;
      if (2 * i < rows) gstore(reinterpret_cast<uint4*>(o), lo);
      if (2 * i + 1 < rows) gstore(reinterpret_cast<uint4*>(o + pitch), hi);
    }
  }
}

constexpr float kBf16Round = 0x1.ffp+127f;  // the smallest value that bf16 rounds to infinity

// Three bf16 pairs whose sum is two fp32 values to 2^-25 of each: rounded, the
// rest rounded, the rest of that.
__device__ __forceinline__ void split3(float a, float b, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; i++) {
    p[i] = bf16x2_rn(a, b);
    a -= __uint_as_float(p[i] << 16);
    b -= __uint_as_float(p[i] & 0xFFFF0000u);
  }
}

// The adapters' share of a warp's 32 features x 32 rows (features n0 .., rows
// row .. row + nc - 1): sum_r u[row][r] b[id][n][r], on the bf16 tensor cores, 16
// features x 8 rows x 16 ranks an instruction. u is fp32: three bf16 terms of it
// (2^-25 of u) multiply b and meet in the fp32 accumulator; a bf16 result, whose
// own rounding is 2^-8, takes two (2^-17; a third takes a decode step of 64 adapters
// from 22.6 to 24.6 us). Each distinct adapter of the rows is one pass over the 8-row
// blocks that use it, with the other rows' u as zeros -- which add nothing while b is
// finite, so a row's result does not depend on its neighbours; the next pass's b is
// loaded meanwhile. A pass whose b (these features, these ranks) holds an infinity or
// NaN, which 0 would not cancel, is left out, and so is a row whose u holds an infinity
// or a value that bf16 rounds to one (split3 would give inf - inf; a NaN stays one):
// `slow` returns those rows, their sums zero, for add_slow(). The ranks are numbered as
// a lane loads them (8 of a row, 16 bytes), alike on both sides. Reads nothing of
// the projection, so a tile's first chunk is summed while the tile is still being
// multiplied. What bounds it: these instructions wait behind the projection's
// tcgen05 ones, about 100 cycles each, so the fewer the better. In fp32 FMAs, with
// u read from shared memory, 8192 rows at rank 32 took 191 us against 147.
// acc[m][j][e]: feature 16 m + 8 (e / 2) + lane / 4, row 8 j + 2 (lane % 4) + e % 2.
__device__ __forceinline__ void sum_adapters(float (&acc)[2][4][4], uint32_t& slow, const GemmArgs& a, int64_t row,
                                             int64_t n0, int features, int nc, int lane) {
  slow = 0;
#pragma unroll
  for (int m = 0; m < 2; m++)
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) acc[m][j][e] = 0.0f;
  int32_t id = lane < nc ? gload(&a.ids[row + lane]) : -1;
  if (id < 0 || id >= a.adapters) id = -1;
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
  const uint32_t all = __ballot_sync(0xFFFFFFFFu, id >= 0 && __ffs(same) - 1 == lane);
  if (all == 0) return;
  const uint32_t live = __ballot_sync(0xFFFFFFFFu, id >= 0);
  const int gr = lane >> 2, q8 = (lane & 3) * 8;
  const int64_t pitch = static_cast<int64_t>(a.ni) * a.rank;
  const uint16_t* b = a.b + (n0 + gr) * a.rank + q8;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
  for (int r = 0; r < a.rank; r += 32) {
    uint4 w[2][2], wn[2][2];  // features 16 m + 8 h + gr, ranks r + q8 .. + 7
    auto load_b = [&](int32_t i, uint4(&v)[2][2]) {
#pragma unroll
      for (int m = 0; m < 2; m++)
#pragma unroll
        for (int h = 0; h < 2; h++)
          v[m][h] = r + q8 < a.rank && 16 * m + 8 * h + gr < features
                        ? gload(reinterpret_cast<const uint4*>(b + i * pitch + (16 * m + 8 * h) * a.rank + r))
                        : zero;
    };
    uint32_t firsts = all;
    int32_t cur = __shfl_sync(0xFFFFFFFFu, id, __ffs(firsts) - 1);
    firsts &= firsts - 1;
    load_b(cur, w);
    float4 u[4][2];  // row 8 j + gr, ranks r + q8 .. + 7
    float largest = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      u[j][0] = u[j][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (((live >> (8 * j + gr)) & 1) && r + q8 < a.rank) {
        const float4* up = reinterpret_cast<const float4*>(a.u + (row + 8 * j + gr) * a.rank + r + q8);
        u[j][0] = gload(up);
        u[j][1] = gload(up + 1);
      }
      largest = fmaxf(largest, fmaxf(fmaxf(fmaxf(fabsf(u[j][0].x), fabsf(u[j][0].y)), fmaxf(fabsf(u[j][0].z), fabsf(u[j][0].w))),
                                     fmaxf(fmaxf(fabsf(u[j][1].x), fabsf(u[j][1].y)), fmaxf(fabsf(u[j][1].z), fabsf(u[j][1].w)))));
    }
    if (__any_sync(0xFFFFFFFFu, largest >= kBf16Round)) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        bool high = false;
#pragma unroll
        for (int h = 0; h < 2; h++)
          high = high || fabsf(u[j][h].x) >= kBf16Round || fabsf(u[j][h].y) >= kBf16Round || fabsf(u[j][h].z) >= kBf16Round ||
                 fabsf(u[j][h].w) >= kBf16Round;
        uint32_t rows = __ballot_sync(0xFFFFFFFFu, high);  // lane 4 gr + q: row gr
        rows |= rows >> 1;
        rows |= rows >> 2;  // bit 4 gr: any of the row's four lanes
        if ((rows >> (lane & 28)) & 1) u[j][0] = u[j][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < 8; k++) slow |= ((rows >> (4 * k)) & 1u) << (8 * j + k);
      }
    }
#pragma unroll 1
    while (true) {
      const bool more = firsts != 0;
      const int32_t nxt = __shfl_sync(0xFFFFFFFFu, id, more ? __ffs(firsts) - 1 : 0);
      firsts &= firsts - 1;
      if (more) load_b(nxt, wn);
      const uint32_t users = __ballot_sync(0xFFFFFFFFu, id == cur);
      uint32_t top = 0;  // the largest exponent and mantissa of each half word
#pragma unroll
      for (int m = 0; m < 2; m++)
#pragma unroll
        for (int h = 0; h < 2; h++)
          top = umax2(umax2(umax2(top, w[m][h].x & 0x7FFF7FFFu), umax2(w[m][h].y & 0x7FFF7FFFu, w[m][h].z & 0x7FFF7FFFu)),
                      w[m][h].w & 0x7FFF7FFFu);
      const bool finite = !__any_sync(0xFFFFFFFFu, (top & 0xFFFFu) >= 0x7F80u || top >= 0x7F800000u);
      if (!finite) slow |= users;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (!finite || ((users >> (8 * j)) & 0xFF) == 0) continue;
        const bool mine = (users >> (8 * j + gr)) & 1;
        const float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float4 u0 = mine ? u[j][0] : z, u1 = mine ? u[j][1] : z;
        uint32_t p[4][3];
        split3(u0.x, u0.y, p[0]);
        split3(u0.z, u0.w, p[1]);
        split3(u1.x, u1.y, p[2]);
        split3(u1.z, u1.w, p[3]);
#pragma unroll
        for (int i = 2; i >= 0; i--) {
          if (i == 2 && !a.out_f32) continue;
#pragma unroll
          for (int m = 0; m < 2; m++) {
            mma_bf16(acc[m][j], w[m][0].x, w[m][1].x, w[m][0].y, w[m][1].y, p[0][i], p[1][i]);
            mma_bf16(acc[m][j], w[m][0].z, w[m][1].z, w[m][0].w, w[m][1].w, p[2][i], p[3][i]);
          }
        }
      }
      if (!more) break;
      cur = nxt;
#pragma unroll
      for (int m = 0; m < 2; m++)
#pragma unroll
        for (int h = 0; h < 2; h++) w[m][h] = wn[m][h];
    }
  }
  if (slow) {
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          if ((slow >> (8 * j + 2 * (lane & 3) + (e & 1))) & 1) acc[m][j][e] = 0.0f;
  }
}

// y2[i] (lane = feature, rows 2i and 2i + 1) += acc, which changes layout in
// shared memory, 16 rows at a time: [row][feature], the features' blocks of 8
// exchanged by row pair so that an instruction's four row pairs lie in different banks.
__device__ __forceinline__ void add_adapters(uint64_t (&y2)[16], uint32_t (&turn)[16][32], const float (&acc)[2][4][4],
                                             int lane) {
  const int gr = lane >> 2, q8 = (lane & 3) * 8;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    __syncwarp();
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          turn[8 * j + (q8 >> 2) + (e & 1)][(16 * m + 8 * (e >> 1) + gr) ^ q8] = __float_as_uint(acc[m][2 * h + j][e]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const int f = lane ^ ((k & 3) << 3);
      uint64_t& y = y2[8 * h + k];
      y = pack2(lo2(y) + __uint_as_float(turn[2 * k][f]), hi2(y) + __uint_as_float(turn[2 * k + 1][f]));
    }
  }
}

// The rows that sum_adapters() left out, y2 as there: fp32 FMAs in the order of the ranks,
// a lane a feature. Infinities and NaN come out as the formula has them; the
// rows' finite results are exact to the FMAs' roundings. The other rows add -0.
__device__ __forceinline__ void add_slow(uint64_t (&y2)[16], uint32_t (&turn)[16][32], uint32_t slow, const GemmArgs& a,
                                         int64_t row, int64_t n, bool live, int lane) {
#pragma unroll
  for (int h = 0; h < 2; h++) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; i++) turn[i][lane] = 0x80000000u;
    for (uint32_t left = (slow >> (16 * h)) & 0xFFFFu; left != 0; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const int64_t t = row + 16 * h + i, id = gload(&a.ids[t]);
      const float* u = a.u + t * a.rank;
      const uint16_t* b = a.b + (id * a.ni + n) * a.rank;
      float s = 0.0f;
#pragma unroll 1
      for (int r = 0; live && r < a.rank; r++)
        s = __fmaf_rn(gload(u + r), __uint_as_float(static_cast<uint32_t>(gload(b + r)) << 16), s);
      turn[i][lane] = __float_as_uint(s);
    }
#pragma unroll
    for (int k = 0; k < 8; k++) {
      uint64_t& y = y2[8 * h + k];
      y = pack2(lo2(y) + __uint_as_float(turn[2 * k][lane]), hi2(y) + __uint_as_float(turn[2 * k + 1][lane]));
    }
  }
}

// One stage's scale copies and MMAs, by one thread. All descriptors are one
// base plus constants and the full stage is unrolled: an operand built per
// instruction costs about 70 cycles of issue for each copy or MMA, more than the
// 128 cycles an N = 256 MMA runs (measured: 12 copies and 4 MMAs 1070 cycles
// a stage so, 513 as here, which is the MMAs alone).
template <bool kGated, bool kPair, bool kFull>
__device__ __forceinline__ void issue_stage(uint32_t st, uint32_t tmem, uint32_t acc, uint32_t idesc, int ksteps,
                                            bool two, bool first) {
  using Stage = GemmStage<kGated>;
  constexpr int kTileUnits = kGScaleTile >> 4;
  constexpr int kJCols = kGated ? 4 : 8;
  const uint64_t di = mma_desc(st), dj = mma_desc(st + Stage::kIData);
  const uint64_t si = scale_desc(st + Stage::kData), sj = scale_desc(st + Stage::kData + Stage::kISf);
  const uint32_t ti = tmem + kGSfCol, tj = ti + (kGated ? 32 : 16);
#pragma unroll
  for (int k = 0; k < 4; k++)
    if (kFull || k < ksteps) {
      tmem_copy_scales<kPair>(ti + 4 * k, si + kTileUnits * k);
      if (kGated) tmem_copy_scales<kPair>(ti + 16 + 4 * k, si + kTileUnits * (4 + k));
      tmem_copy_scales<kPair>(tj + kJCols * k, sj + kTileUnits * k);
    }
  if (!kGated && two) {
#pragma unroll
    for (int k = 0; k < 4; k++)
      if (kFull || k < ksteps) tmem_copy_scales<kPair>(tj + 8 * k + 4, sj + kTileUnits * (4 + k));
  }
#pragma unroll
  for (int k = 0; k < 4; k++)
    if (kFull || k < ksteps) {
      mma_nvf4<kPair>(acc, di + 2 * k, dj + 2 * k, idesc, ti + 4 * k, tj + kJCols * k, !first || k > 0);
      if (kGated)
        mma_nvf4<kPair>(acc + 128, di + (kGIBytes >> 4) + 2 * k, dj + 2 * k, idesc, ti + 16 + 4 * k, tj + kJCols * k,
                        !first || k > 0);
    }
}

// ------------------------------------------------------------------ kernel

template <class Routing, int kMode, bool kTma, bool kPair>
__global__ void __launch_bounds__(kGThreads, 1)
group_gemm_kernel(const __grid_constant__ Routing routing, const __grid_constant__ CUtensorMap imap,
                  const __grid_constant__ CUtensorMap jmap, const __grid_constant__ CUtensorMap jmap_small,
                  const __grid_constant__ GemmArgs a) {
  constexpr bool kGated = kMode == kGemmGated;
  using Stage = GemmStage<kGated>;
  using Walk = GemmWalk<kMode, kPair>;
  constexpr int kStages = Stage::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  GemmSmem<kGated>& sm = *reinterpret_cast<GemmSmem<kGated>*>(base);
  int32_t* off = reinterpret_cast<int32_t*>(base + ((sizeof(GemmSmem<kGated>) + 15) & ~size_t{15}));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(blockIdx.x & 1) : 0;  // in the pair

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; s++) {
      mbar_init(&sm.full[s], (a.producer ? 1 : 0) + (a.loaders ? 1 : 0));
      mbar_init(&sm.peer_full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.acc_full, 1);
    mbar_init(&sm.acc_free, kGEpiWarps * (kPair ? 2 : 1));
    mbar_init(&sm.drain, 1);
    sm.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    tmem_alloc<kPair>(&sm.tmem);
    tc_fence_before();
  }
  routing.load(sm.routing, off);  // ends with a __syncthreads
  if (kPair) pair_sync();         // the other CTA's barriers are initialised, its tensor memory allocated
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sm.tmem);

  if (warp < kGLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGRegsIssue));
    if (!sm.routing.ok) {
      // nothing to do
    } else if (warp == 0 && a.producer) {
      Walk walk(sm.routing, a);
      GemmTile t;
      const bool elected = elect_one();
      GemmRing<kStages> ring;
      uint32_t n = 0;
      bool ok = true;
      const uint64_t pol = policy_evict_normal();
      while (ok && walk.next(t)) {
        const int nkb = (t.kc + kGK - 1) / kGK;
        // this CTA's J rows: boxes of 128, the rest in boxes of 32
        const int jrows = kPair ? ((t.jv + 31) & ~31) / 2 : t.jv;
        const int big = jrows / kGBigJ, small = (jrows - big * kGBigJ + kGBoxJ - 1) / kGBoxJ;
        const int jblocks = (t.jv + 127) / 128;
        const int64_t kt = t.kc / 64;
        // tiled scales: tile (row block, k step) at (block * kc/64 + step) * 512
        const uint8_t* is = a.i.scale + (kMode == kGemmWgrad ? t.goff * a.ni / 16 + t.i0 / 128 * kt * kGScaleTile
                                                             : t.irow / 128 * kt * kGScaleTile);
        const uint8_t* js = a.j.scale + (kMode == kGemmWgrad ? t.goff * a.nj / 16 + t.j0 / 128 * kt * kGScaleTile
                                                             : t.jrow / 128 * kt * kGScaleTile);
        const int iy = static_cast<int>(t.irow), jy = static_cast<int>(t.jrow) + rank * jrows;
        uint32_t data_bytes = 0, tiles = 0;
        if (kTma) data_bytes = (kGated ? 2 : 1) * kGIBytes + (big * kGBigJ + small * kGBoxJ) * 128;
        if (a.i.tiled) tiles += kGated ? 2 : 1;
        if (a.jbulk) tiles += jblocks;
        for (int kb = 0; kb < nkb; kb++, n++, ring.next()) {
          const uint32_t s = ring.s;
          if (!mbar_wait(&sm.empty[s], ring.phase ^ 1)) {
            ok = false;
            break;
          }
          if (elected) {
            uint8_t* st = sm.stage[s];
            uint64_t* bar = &sm.full[s];
            const uint32_t sf_bytes = min(4, (t.kc - kb * kGK + 63) / 64) * kGScaleTile;
            mbar_expect_tx(bar, data_bytes + tiles * sf_bytes);
            if (kTma) {
              tma_load_2d(st, &imap, kb * 128, iy, bar, pol);
              if (kGated) tma_load_2d(st + kGIBytes, &imap, kb * 128, iy + a.ni, bar, pol);
              for (int b = 0; b < big; b++)
                tma_load_2d(st + Stage::kIData + b * kGBigJ * 128, &jmap, kb * 128, jy + b * kGBigJ, bar, pol);
              for (int b = 0; b < small; b++)
                tma_load_2d(st + Stage::kIData + (big * kGBigJ + b * kGBoxJ) * 128, &jmap_small, kb * 128,
                            jy + big * kGBigJ + b * kGBoxJ, bar, pol);
            }
            uint8_t* sf = st + Stage::kData;
            const int64_t so = static_cast<int64_t>(kb) * 4 * kGScaleTile;
            if (a.i.tiled) {
              bulk_load(sf, is + so, sf_bytes, bar);
              if (kGated) bulk_load(sf + 4 * kGScaleTile, is + a.ni / 128 * kt * kGScaleTile + so, sf_bytes, bar);
            }
            if (a.jbulk)
              for (int b = 0; b < jblocks; b++)
                bulk_load(sf + Stage::kISf + b * 4 * kGScaleTile, js + b * kt * kGScaleTile + so, sf_bytes, bar);
          }
          __syncwarp();
        }
      }
      if (!ok) {
        sm.gave_up = 1;
        for (uint32_t k = n > kStages ? n - kStages : 0; k < n; k++)
          mbar_wait(&sm.full[k % kStages], (k / kStages) & 1);
      }
    } else if (warp == 1 && rank == 1) {
      // second CTA of a pair: tells the first that a stage is full
      GemmBlocks<kMode, kPair> at(sm.routing, a);
      const bool elected = elect_one();
      GemmRing<kStages> ring;
      for (; at.more; at.next(), ring.next()) {
        if (!mbar_wait(&sm.full[ring.s], ring.phase)) {
          sm.gave_up = 1;
          break;
        }
        if (elected) mbar_arrive_first(&sm.peer_full[ring.s]);
        __syncwarp();
      }
    } else if (warp == 1) {
      Walk walk(sm.routing, a);
      GemmTile t;
      const bool elected = elect_one();
      GemmRing<kStages> ring;
      uint32_t tiles = 0;
      bool ok = true;
      const uint32_t stages = smem_addr(sm.stage[0]);
      while (ok && walk.next(t)) {
        const int nkb = (t.kc + kGK - 1) / kGK;
        if (nkb == 0) continue;
        if (tiles > 0 && !mbar_wait(&sm.acc_free, (tiles - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + ((tiles & 1) ? kGAcc1 : 0);
        const int cols = kPair ? (t.jv + 31) & ~31 : (t.jv + 15) & ~15;
        const uint32_t idesc = mma_idesc<kPair>(cols);
        for (int kb = 0; kb < nkb; kb++, ring.next()) {
          const uint32_t s = ring.s;
          if (!mbar_wait(&sm.full[s], ring.phase) || (kPair && !mbar_wait(&sm.peer_full[s], ring.phase))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int ksteps = min(4, (t.kc - kb * kGK + 63) / 64);
          if (elected) {
            const uint32_t st = stages + s * Stage::kBytes;
            if (ksteps == 4)
              issue_stage<kGated, kPair, true>(st, tmem, acc, idesc, 4, cols > 128, kb == 0);
            else
              issue_stage<kGated, kPair, false>(st, tmem, acc, idesc, ksteps, cols > 128, kb == 0);
            mma_commit<kPair>(&sm.empty[s]);
          }
          __syncwarp();
        }
        if (ok && elected) mma_commit<kPair>(&sm.acc_full);
        __syncwarp();
        tiles++;
      }
      if (!ok) {
        sm.gave_up = 1;
        if (elected) mma_commit<kPair>(&sm.drain);
        __syncwarp();
        mbar_wait(&sm.drain, 0);
      }
    }
  } else if (warp < kGEpiWarp) {
    if (sm.routing.ok && a.loaders) {
      // Each of the four warps fills every fourth stage by itself, so that four
      // stages' latencies overlap.
      GemmBlocks<kMode, kPair> at(sm.routing, a);
      GemmRing<kStages> ring;
      bool ok = true;
      // Rows lane + 32 e of each 128-row block of scales (I, then two of J; gated:
      // gate, up, J), read ahead as they are; p: the next block's, row lane.
      constexpr int kJ = kGated ? 2 : 1;
      struct Rows {
        uint32_t w[3][4][5];
      };
      Rows r;
      // of a tile's J rows, those that read() reads
      auto whole_rows = [&](const GemmTile& t) {
        return kMode == kGemmWgrad ? t.jv : min(t.jv, a.j_whole - static_cast<int32_t>(t.jrow));
      };
      auto read = [&] {
        const GemmTile& t = at.t;
        const int32_t cols = t.kc / 16, first = at.kb * 16, left = cols - first;
        const int how = (cols & 15) == 0 ? kRead16 : (cols & 3) == 0 ? kReadWords : kReadBytes;
        if (!a.i.tiled) {
          const int64_t ib = kMode == kGemmWgrad ? t.goff * a.ni / 16 + static_cast<int64_t>(t.i0) * cols : t.irow * cols;
          const uint8_t* p = a.i.scale + ib + static_cast<int64_t>(lane) * cols + first;
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const bool in = lane + 32 * e < t.iv;
            const uint8_t* pe = p + static_cast<int64_t>(32 * e) * cols;
            read_scales(in ? pe : nullptr, how, left, r.w[0][e]);
            if (kGated) read_scales(in ? pe + static_cast<int64_t>(a.ni) * cols : nullptr, how, left, r.w[1][e]);
          }
        }
        if (!a.jbulk) {
          const int64_t jb = kMode == kGemmWgrad ? t.goff * a.nj / 16 : (t.jrow - t.j0) * cols;  // the group's first row
          const int jv = whole_rows(t);
#pragma unroll
          for (int h = 0; h < (kGated ? 1 : 2); h++) {
            if (128 * h >= t.jv) break;
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const int j = lane + 32 * e + 128 * h, jr = t.j0 + j;
              const uint8_t* pe;
              if (a.j.tiled)  // a J tile inside a 128-row block (jt < 128): its rows out of the block's tiles; the
                              // scales in tensor memory cannot start at a later column
                pe = a.j.scale + jb + (static_cast<int64_t>(jr >> 7) * (cols >> 2) + at.kb * 4) * kGScaleTile +
                     (jr & 31) * 16 + ((jr & 127) >> 5) * 4;
              else
                pe = a.j.scale + jb + static_cast<int64_t>(jr) * cols + first;
              read_scales(j < jv ? pe : nullptr, a.j.tiled ? kReadTiled : how, left, r.w[kJ + h][e]);
            }
          }
        }
      };
      // Words out of what was read raw: the rows' first bytes as read() found them.
      auto words = [&](int k, int64_t row, bool tiled) {
        const int32_t cols = at.t.kc / 16;
        if (tiled || (cols & 15) == 0) return;
#pragma unroll
        for (int e = 0; e < 4; e++)
          scale_words((cols & 3) == 0 ? 0u : static_cast<uint32_t>((row + lane + 32 * e) * cols & 3) * 8, cols - at.kb * 16,
                      r.w[k][e]);
      };
      auto skip = [&](int n) {
        for (int k = 0; k < n && at.more; k++) at.next();
      };
      const int mine = warp - kGLoadWarp;
      skip(mine);
      ring.s = mine;
      if (at.more) read();
      while (at.more) {
        const uint32_t s = ring.s;
        if (!mbar_wait(&sm.empty[s], ring.phase ^ 1)) {
          ok = false;
          break;
        }
        uint8_t* st = sm.stage[s];
        const GemmTile& t = at.t;
        // the rows whose offsets decide the first byte (a group of wgrad starts on 16 bytes)
        const int64_t i_row = kMode == kGemmWgrad ? t.i0 : t.irow, j_row = kMode == kGemmWgrad ? t.j0 : t.jrow;
        if (!kTma) {
          const int64_t row_bytes = t.kc / 2;
          const uint8_t *ic, *jc;
          if (kMode == kGemmWgrad) {
            ic = a.i.data + t.goff * a.ni / 2 + t.i0 * row_bytes;
            jc = a.j.data + t.goff * a.nj / 2 + t.j0 * row_bytes;
          } else {
            ic = a.i.data + t.irow * row_bytes;
            jc = a.j.data + t.jrow * row_bytes;
          }
          const uint32_t d = smem_addr(st);
          // this CTA's J rows
          const int cols = kPair ? ((t.jv + 31) & ~31) / 2 : (t.jv + 15) & ~15, kbyte = at.kb * 128;
          const int jv = max(0, min(cols, t.jv - rank * cols));
          if (jv > 0) jc += rank * cols * row_bytes;
          if (row_bytes % 16 == 0) {
            load_codes<16>(d, ic, row_bytes, kGI, t.iv, kbyte, lane);
            if (kGated) load_codes<16>(d + kGIBytes, ic + a.ni * row_bytes, row_bytes, kGI, t.iv, kbyte, lane);
            load_codes<16>(d + Stage::kIData, jc, row_bytes, cols, jv, kbyte, lane);
          } else {
            load_codes<8>(d, ic, row_bytes, kGI, t.iv, kbyte, lane);
            if (kGated) load_codes<8>(d + kGIBytes, ic + a.ni * row_bytes, row_bytes, kGI, t.iv, kbyte, lane);
            load_codes<8>(d + Stage::kIData, jc, row_bytes, cols, jv, kbyte, lane);
          }
          cp_async_commit();
        }
        uint8_t* sf = st + Stage::kData;
        if (!a.i.tiled) {
          words(0, i_row, false);
          store_scales(sf, lane, r.w[0]);
          if (kGated) {
            words(1, i_row + a.ni, false);
            store_scales(sf + 4 * kGScaleTile, lane, r.w[1]);
          }
        }
        if (!a.jbulk) {
          words(kJ, j_row, a.j.tiled);
          store_scales(sf + Stage::kISf, lane, r.w[kJ]);
          if (!kGated && t.jv > 128) {
            words(2, j_row + 128, a.j.tiled);
            store_scales(sf + Stage::kISf + 4 * kGScaleTile, lane, r.w[2]);
          }
          const int jw = whole_rows(t);
          if (jw < t.jv) {
            const int32_t cols = t.kc / 16, j0 = max(jw, 0), first = at.kb * 16;
            patch_scales(sf + Stage::kISf, a.j.scale + (t.jrow + j0) * cols + first, cols, cols - first, j0, t.jv, lane);
          }
        }
        if (!kTma) cp_async_wait<0>();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[s]);
        skip(4);
        ring.s += 4;
        if (ring.s >= kStages) {
          ring.s -= kStages;
          ring.phase ^= 1;
        }
        if (at.more) read();
      }
      cp_async_wait<0>();
      if (!ok) sm.gave_up = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGRegsEpi));
    if (sm.routing.ok) {
      const int q = warp & 3;                       // accumulator lanes 32q .. 32q+31
      const int half = (warp - kGEpiWarp) >> 2;     // chunks of parity `half`
      const int il = 32 * q + lane;
      // chunks of 32 columns; the first one a warp takes holds its part of
      // the columns both accumulators share (set 0: the last two, set 1: the
      // first two; gated: of the up or the gate half)
      constexpr int kChunks = kGated ? 4 : 8, kMine = kChunks / 2;
      auto chunk = [&](int set, int ci) { return (set == 0 ? (ci == 0 ? kChunks - 2 : 2 * (ci - 1)) : 2 * ci) + half; };
      // first column of a warp's ci-th chunk and its rows (adapters: a tile of a few
      // rows is cut in two, so that a decode step's adapters are shared out)
      auto first_col = [&](const GemmTile& t, int set, int ci) {
        const int c = chunk(set, ci);
        return kMode == kGemmAdapter && t.jv <= 32 && c < 2 ? c * (((t.jv + 15) >> 4) << 3) : 32 * c;
      };
      auto chunk_rows = [&](const GemmTile& t) {
        return kMode == kGemmAdapter && t.jv <= 32 ? ((t.jv + 15) >> 4) << 3 : 32;
      };
      // a tile's factors, read before the tile before it is finished
      struct Factors {
        float i, up;
        float j[kMine];
      };
      auto read = [&](const GemmTile& t, int set, Factors& f) {
        f.i = f.up = 0.0f;
        if (il < t.iv) {
          f.i = gload(&a.i.s2[t.irow + il]);
          if (kGated) f.up = gload(&a.i.s2[t.irow + a.ni + il]);
        }
#pragma unroll
        for (int ci = 0; ci < kMine; ci++) {
          const int c = first_col(t, set, ci) + lane;
          f.j[ci] = c < t.jv ? gload(&a.j.s2[t.jrow + c]) : 0.0f;
        }
      };
      Walk walk(sm.routing, a);
      GemmTile t, t1;
      Factors f{}, f1{};
      uint32_t tiles = 0;
      bool more = walk.next(t1);
      if (more && t1.kc > 0) read(t1, 0, f1);
      float* sjw = sm.sj[warp - kGEpiWarp];
      uint32_t(&turn)[16][32] = sm.turn[warp - kGEpiWarp];
      while (more) {
        t = t1;
        f = f1;
        const bool empty = t.kc == 0;
        more = walk.next(t1);
        f1 = Factors{};
        if (more && t1.kc > 0) read(t1, (tiles + (empty ? 0 : 1)) & 1, f1);
        const bool live = il < t.iv;
        const int64_t n = t.i0 + il;
        const int set = tiles & 1;
        const uint32_t acc = tmem + (set ? kGAcc1 : 0) + (static_cast<uint32_t>(32 * q) << 16);
        const uint64_t si2 = pack2(f.i, f.i), su2 = pack2(f.up, f.up);
        bool freed = empty, full = empty, ok = true, no_shared = false;
        auto release = [&] {
          if (!freed) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (kPair)
                mbar_arrive_first(&sm.acc_free);
              else
                mbar_arrive(&sm.acc_free);
            }
            freed = true;
          }
        };
        // The accumulator is waited for when it is first read. Every warp waits for
        // every tile's, and frees the shared columns only after that: freed
        // before, the next tile's MMAs could complete a second phase of acc_full,
        // and a warp that still waits for this one's would wait for good.
        auto wait_full = [&] {
          if (!full) {
            ok = mbar_wait(&sm.acc_full, tiles & 1);
            full = true;
            tc_fence_after();
            if (no_shared) release();
          }
        };
        if (kMode == kGemmAdapter)
          grid_dependency_wait();  // u comes from the kernel before this one
        else
          wait_full();
#pragma unroll 1
        for (int ci = 0; ci < kMine && ok; ci++) {
          const int c0 = first_col(t, set, ci);
          if (c0 >= t.jv) {
            if (ci == 0) {  // no columns of this warp's among the shared ones
              if (full)
                release();
              else
                no_shared = true;
            }
            continue;
          }
          const int nc = min(chunk_rows(t), t.jv - c0);
          const int64_t row = t.jrow + c0;
          const int features = t.iv - 32 * q;
          float extra[2][4][4];
          uint32_t slow = 0;
          if (kMode == kGemmAdapter) {
            sum_adapters(extra, slow, a, row, t.i0 + 32 * q, features, nc, lane);
            wait_full();
          }
          uint32_t v[32], w[32];
          if (empty) {
#pragma unroll
            for (int k = 0; k < 32; k++) v[k] = w[k] = 0;
          } else {
            tmem_load32(acc + c0, v);
            if (kGated) tmem_load32(acc + 128 + c0, w);
          }
          float fj = f.j[0];
#pragma unroll
          for (int k = 1; k < kMine; k++)
            if (ci == k) fj = f.j[k];
          __syncwarp();  // the previous chunk's factors have been read
          sjw[lane] = empty ? 0.0f : fj;
          __syncwarp();
          if (!empty) {
            tmem_load_wait(v);
            if (kGated) tmem_load_wait(w);
          }
          if (ci == 0) release();
          uint64_t y[16], z[16];  // rows 2k and 2k + 1
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float4 s = *reinterpret_cast<const float4*>(sjw + 2 * k);
            const uint64_t s0 = pack2(s.x, s.y), s1 = pack2(s.z, s.w);
            y[k] = mul2x(mul2x(pair2(v[2 * k], v[2 * k + 1]), s0), si2);
            y[k + 1] = mul2x(mul2x(pair2(v[2 * k + 2], v[2 * k + 3]), s1), si2);
            if (kGated) {
              z[k] = mul2x(mul2x(pair2(w[2 * k], w[2 * k + 1]), s0), su2);
              z[k + 1] = mul2x(mul2x(pair2(w[2 * k + 2], w[2 * k + 3]), s1), su2);
            }
          }
          uint32_t b[16];
          if (kGated) {
            if (a.pre != nullptr) {
              const int64_t pitch = 2 * static_cast<int64_t>(a.ni);
              uint16_t* p = a.pre + row * pitch + t.i0 + 32 * q;
#pragma unroll
              for (int k = 0; k < 16; k++) b[k] = bf16_pair(y[k]);
              store_bf16(b, turn, p, pitch, nc, features, lane);
#pragma unroll
              for (int k = 0; k < 16; k++) b[k] = bf16_pair(z[k]);
              store_bf16(b, turn, p + a.ni, pitch, nc, features, lane);
            }
#pragma unroll
            for (int k = 0; k < 16; k++) b[k] = bf16_pair(silu_times2(y[k], z[k]));
            store_bf16(b, turn, static_cast<uint16_t*>(a.out) + row * a.ni + t.i0 + 32 * q, a.ni, nc, features, lane);
          } else {
            if (kMode == kGemmAdapter) {
              add_adapters(y, turn, extra, lane);
              if (slow != 0) add_slow(y, turn, slow, a, row, n, live, lane);
            }
            if (a.out_f32) {
              float* o = static_cast<float*>(a.out) + row * a.ni + n;
#pragma unroll
              for (int k = 0; k < 32; k++) {
                if (k < nc && live) gstore(o, k & 1 ? hi2(y[k >> 1]) : lo2(y[k >> 1]));
                o += a.ni;
              }
            } else {
#pragma unroll
              for (int k = 0; k < 16; k++) b[k] = bf16_pair(y[k]);
              store_bf16(b, turn, static_cast<uint16_t*>(a.out) + row * a.ni + t.i0 + 32 * q, a.ni, nc, features, lane);
            }
          }
        }
        wait_full();
        if (!ok) {
          if (lane == 0) sm.gave_up = 1;
          break;
        }
        if (!empty) tiles++;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (kPair) pair_sync();  // the other CTA reads this one's stages and arrives on its barriers until here
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<kPair>(tmem);
  }
  if (threadIdx.x == 0 && sm.gave_up) {
    routing.report(NVFP4_ERR_TIMEOUT);
    if (kMode == kGemmAdapter && a.status != nullptr) gstore(a.status, static_cast<int32_t>(NVFP4_ERR_TIMEOUT));
  }
}

}  // namespace nvfp4rs
