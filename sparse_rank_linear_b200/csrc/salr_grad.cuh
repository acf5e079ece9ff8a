// salr_grad.cuh - the gradients of the layer Y = X W^T + (X A) B for a frozen W:
//
//     u = dY B^T        dX = dY W + u A^T        dA = X^T u
//     t = X A                                    dB = t^T dY
//
// Three launches after the weight has been expanded to a dense bf16 N x K scratch, all
// tcgen05 products of operand tiles that TMA brings in as they lie in memory: an operand
// whose reduction index is its row index is read MN-major (transposed by the tensor core),
// so nothing is transposed in memory.
//
// The launches overlap at their ends (programmatic dependent launch): each kernel starts as
// the SMs of the one before it fall free, and waits for it where it reads its results.
//
// 1. grad_skinny_kernel, t and u in one launch (two problems): 128 tokens x all ranks per
//    CTA, the reduction over K or N split over CTAs.  The fp32 result is stored as two bf16
//    parts side by side, hi = bf16(t) and lo = bf16(t - hi), so that the next products take
//    t and u to 16 bits of significand and dX, dA and dB carry no rounding but their own.
// 2. grad_dx_kernel: dX, by pairs of CTAs (cta_group::2).  The u A^T term runs as extra
//    reduction steps of the same accumulator.
// 3. grad_skinny_kernel, dA and dB in one launch: 128 rows of K or N x (hi | lo) ranks, the
//    reduction over tokens split over CTAs; the two halves are added in the epilogue.
//
// Parts of a split reduction are added up in a fixed order: results repeat bit for bit.
//
// Bounds: 2 is tensor-bound (2 M N K flops): 2.44 ms alone for N = 28672, K =
// 8192, M = 8192, 1.58 PFLOP/s, and 2.93 in a long run under the power cap.  1 and 3 read X and dY
// once each and are bound by HBM or, when X and dY stay in L2, by L2: 132 and 137 us for those
// sizes (604 MB, 94 us at the copy rate).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "sm100.cuh"

namespace salr {

// The next 1024-byte boundary of shared memory, by an offset: rounding the pointer itself
// would hide from the compiler that it is shared memory, and cost 64-bit addresses and
// generic loads.
__device__ __forceinline__ uint8_t* align_1024(uint8_t* p) { return p + ((0u - smem_u32(p)) & 1023u); }

// ---------------------------------------------------------------- CTA-pair wrappers

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of shared-memory location `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// mbar_wait for a barrier that the other CTA of the pair arrives on.
__device__ __forceinline__ bool mbar_wait_pair(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 255u) == 255u && clock64() - t0 > wait_limit()) return false;
  }
}
// Wait for a copy in flight on the way out after a wait that gave up: 2 ms at most (however
// short the bound on the other waits is, copies land within microseconds, and none may land
// in the shared memory of a CTA that has exited).
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  while (!mbar_try_wait(a, parity) && clock64() - t0 < 4000000) {
  }
}
// Tensor copy into this CTA's shared memory that reports to a barrier of either CTA.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int32_t c0,
                                                 int32_t c1, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar_cluster)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (256 rows, 128 in each CTA's TMEM) (+)= A B^T: each CTA holds its 128 rows of A and its
// half of B's rows at the same shared-memory offsets.  Issued by the pair's first CTA.
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs once every pair MMA issued so far by this thread is done.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// ---------------------------------------------------------------- skinny products

constexpr int kGradThreads = 192;  // warp 0 loads, warp 1 issues MMAs, warps 2-5 epilogue
constexpr int kGradChunk = 64;     // reduction steps per stage

enum : int { GRAD_SPLIT = 0, GRAD_ROWS = 1, GRAD_COLS = 2 };

// C[P x columns] = A-operand (P rows) times B-operand, reduction cut into chunks of 64.
struct GradProblem {
  int tiles, chunks;  // row tiles of 128; chunks of the reduction
  int a_mn, b_mn;     // operand major: 1 if the reduction index is the row index
  int mode;  // GRAD_SPLIT: out[p][c] = hi, out[p][half + c] = lo, row length 2 half
             // GRAD_ROWS:  out[p][c] = column c + column half + c, c < R, row length R
             // GRAD_COLS:  out[c][p] likewise, row length ldo
  int P, R, half, ldo;
  uint16_t* out;
};
struct GradSkinnyParams {
  GradProblem p[2];
  int* status;
  int fail;  // failure tests only: the first CTA leaves out one copy, whose wait then runs out
};

struct GradCtrl {
  uint64_t full[4], empty[4], fin;
  uint32_t tmem;
  int abort;
};

template <int BN>
struct GradSkinny {
  static constexpr int kStage = 16384 + BN * 128;
  // two CTAs an SM up to 128 columns, one with 256
  static constexpr int kStages = BN == 128 ? 3 : 4;
  static constexpr int kSmemBytes = kStages * kStage + 1024 + 256;
  static_assert(kStages * kStage >= (BN + 4) * 512, "the stages hold the fp32 sums at the end");
};

// 16 bytes of shared memory of a CTA of the cluster.
__device__ __forceinline__ float4 ld_cluster4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr));
  return v;
}

// A cluster of `nc` CTAs (1 to 8) takes a row tile, each CTA a part of its reduction.  The
// parts' fp32 sums then lie in the CTAs' shared memory ([row][column], where the stages
// were), and each CTA adds up and writes 128 / nc of the rows, in the order of the parts.
// Parts that met in L2 instead, added up by the last one to arrive, spent most of the time
// in that one CTA's chain of L2 reads: up_proj M = 2048 took 60 + 65 us for the two
// launches.
template <int BN>
__global__ void __launch_bounds__(kGradThreads, BN == 256 ? 1 : 2)
    grad_skinny_kernel(const __grid_constant__ GradSkinnyParams prm, const int nc,
                       const __grid_constant__ CUtensorMap ma0, const __grid_constant__ CUtensorMap mb0,
                       const __grid_constant__ CUtensorMap ma1, const __grid_constant__ CUtensorMap mb1) {
  using L = GradSkinny<BN>;
  extern __shared__ uint8_t smem_raw[];
  // the same offset in every CTA: dynamic shared memory starts alike in all of them
  uint8_t* smem = align_1024(smem_raw);
  GradCtrl* ctrl = reinterpret_cast<GradCtrl*>(smem + L::kStages * L::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x % nc, all = blockIdx.x / nc;
  const int second = all >= prm.p[0].tiles;
  const GradProblem& p = prm.p[second];
  const int tile = all - (second ? prm.p[0].tiles : 0);
  const int c0 = static_cast<int>(static_cast<long long>(part) * p.chunks / nc);
  const int c1 = static_cast<int>(static_cast<long long>(part + 1) * p.chunks / nc);
  const int p0 = tile * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    mbar_init(&ctrl->fin, 1);
    ctrl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&ctrl->tmem, BN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only once this CTA holds its tensor memory: a CTA of the next kernel that came to this SM
  // first could take all of it, and then wait for this grid, which would wait for it.
  griddep_launch_dependents();
  const uint32_t tmem = ctrl->tmem;
  volatile int* abort_flag = &ctrl->abort;

  if (warp == 0) {
    if (lane == 0) {
      const CUtensorMap* ma = second ? &ma1 : &ma0;
      const CUtensorMap* mb = second ? &mb1 : &mb0;
      int s = 0, ph = 0, issued = 0;
      for (int c = c0; c < c1; ++c) {
        if (!mbar_wait(&ctrl->empty[s], ph ^ 1) || *abort_flag) {
          atomicOr(prm.status, DEV_ERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        uint8_t* a = smem + s * L::kStage;
        uint8_t* b = a + 16384;
        uint64_t* bar = &ctrl->full[s];
        mbar_arrive_expect_tx(bar, L::kStage);
        const int r = c * kGradChunk;
        if (p.a_mn) {
          tma_load_2d(a, ma, p0, r, bar);
          tma_load_2d(a + 8192, ma, p0 + 64, r, bar);
        } else if (!prm.fail || blockIdx.x != 0 || c != c0) {
          tma_load_2d(a, ma, r, p0, bar);
        }
        if (p.b_mn) {
#pragma unroll
          for (int h = 0; h < BN / 64; ++h) tma_load_2d(b + h * 8192, mb, h * 64, r, bar);
        } else {
          tma_load_2d(b, mb, r, 0, bar);
        }
        ++issued;
        if (++s == L::kStages) s = 0, ph ^= 1;
      }
      if (*abort_flag)  // let the copies in flight land before the CTA can exit
        for (int i = issued > L::kStages ? issued - L::kStages : 0; i < issued; ++i)
          mbar_drain(&ctrl->full[i % L::kStages], (i / L::kStages) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, BN, p.a_mn, p.b_mn);
      // per 16 reduction steps: 32 bytes along a K-major row, 16 rows of an MN-major tile
      const uint32_t astep = p.a_mn ? 2048 : 32, bstep = p.b_mn ? 2048 : 32;
      const uint32_t albo = p.a_mn ? 8192 : 16, blbo = p.b_mn ? 8192 : 16;
      int s = 0, ph = 0;
      for (int c = c0; c < c1; ++c) {
        if (!mbar_wait(&ctrl->full[s], ph) || *abort_flag) {
          atomicOr(prm.status, DEV_ERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + s * L::kStage), b = a + 16384;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16_ss(tmem, smem_desc_sw128(a + astep * k, albo, 1024),
                      smem_desc_sw128(b + bstep * k, blbo, 1024), idesc, c != c0 || k != 0);
        mma_commit(&ctrl->empty[s]);
        if (++s == L::kStages) s = 0, ph ^= 1;
      }
      mma_commit(&ctrl->fin);
      if (!mbar_wait(&ctrl->fin, 0)) {
        atomicOr(prm.status, DEV_ERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  }
  __syncthreads();  // every product is in TMEM, and the stages are free
  const bool ok = *abort_flag == 0;
  // [128 rows][BN + 4 columns]: with the pad, a quarter-warp's 16-byte accesses fall on
  // different banks both along a row and down a column
  float* sums = reinterpret_cast<float*>(smem);
  constexpr int kRow = BN + 4;
  if (warp >= 2 && ok) {
    const int q = warp & 3;  // TMEM lane quarter
    const uint32_t tm = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float* dst = sums + (32 * q + lane) * kRow;
    tc_fence_after();
    for (int c = 0; c < BN; c += 16) {
      uint32_t v[16];
      tmem_ld16(tm + c, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; e += 4)  // an empty part adds nothing
        *reinterpret_cast<uint4*>(dst + c + e) =
            c1 > c0 ? make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]) : make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync_all();
  if (warp >= 2 && ok) {
    const int rows = 128 / nc, r0 = part * rows, tid = threadIdx.x - 64;
    uint32_t from[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) from[k] = map_to_rank(smem_u32(sums), k < nc ? k : 0);
    // four columns of a row, summed over the parts in order
    auto load4 = [&](int row, int c) {
      const uint32_t at = static_cast<uint32_t>(row * kRow + c) * 4;
      float4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = k < nc ? ld_cluster4(from[k] + at) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 1; k < 8; ++k) x[0].x += x[k].x, x[0].y += x[k].y, x[0].z += x[k].z, x[0].w += x[k].w;
      return x[0];
    };
    auto pack = [](float a, float b) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      return *reinterpret_cast<const uint32_t*>(&h);
    };
    // what a bf16 pair leaves of a and b (nothing of an infinite value: it is all in hi)
    auto rest = [&](uint32_t h, float a, float b) {
      const float h0 = __uint_as_float(h << 16), h1 = __uint_as_float(h & 0xffff0000u);
      return pack(fabsf(h0) <= 3.402823466e38f ? a - h0 : 0.f, fabsf(h1) <= 3.402823466e38f ? b - h1 : 0.f);
    };
    // The sums with hi and lo together.  One with hi that is infinite stands alone: it came from
    // an infinite X or dY, whose product with lo is NaN (lo = 0) or may have the other sign.
    auto whole = [](float hi, float lo) { return fabsf(hi) <= 3.402823466e38f ? hi + lo : hi; };
    if (p.mode == GRAD_COLS) {  // lanes down the rows, which are neighbours in the output
      for (int i = tid; i < rows * (p.R / 4); i += 128) {
        const int row = r0 + i % rows, c = i / rows * 4;
        float4 v = load4(row, c);
        const float4 w = load4(row, p.half + c);
        v = make_float4(whole(v.x, w.x), whole(v.y, w.y), whole(v.z, w.z), whole(v.w, w.w));
        if (p0 + row < p.P) {
          __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.out) + static_cast<size_t>(c) * p.ldo + p0 + row;
          o[0] = __float2bfloat16_rn(v.x);
          o[static_cast<size_t>(p.ldo)] = __float2bfloat16_rn(v.y);
          o[2 * static_cast<size_t>(p.ldo)] = __float2bfloat16_rn(v.z);
          o[3 * static_cast<size_t>(p.ldo)] = __float2bfloat16_rn(v.w);
        }
      }
    } else {  // lanes along the columns
      const int quads = (p.mode == GRAD_SPLIT ? BN : p.R) / 4;
      for (int i = tid; i < rows * quads; i += 128) {
        const int row = r0 + i / quads, c = i % quads * 4;
        const bool live = p0 + row < p.P;
        const size_t pr = static_cast<size_t>(p0) + row;
        // ranks past R are held as zeros: their sums are of zeros, or NaN where an operand is
        // infinite, and a NaN would reach the whole row of dX
        float4 v = c < p.R ? load4(row, c) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.mode == GRAD_SPLIT) {
          const uint32_t h0 = pack(v.x, v.y), h1 = pack(v.z, v.w);
          if (live) {
            uint16_t* o = p.out + pr * 2 * p.half + c;
            *reinterpret_cast<uint2*>(o) = make_uint2(h0, h1);
            *reinterpret_cast<uint2*>(o + p.half) = make_uint2(rest(h0, v.x, v.y), rest(h1, v.z, v.w));
          }
        } else {
          const float4 w = load4(row, p.half + c);
          v = make_float4(whole(v.x, w.x), whole(v.y, w.y), whole(v.z, w.z), whole(v.w, w.w));
          if (live) *reinterpret_cast<uint2*>(p.out + pr * p.R + c) = make_uint2(pack(v.x, v.y), pack(v.z, v.w));
        }
      }
    }
  }
  // this grid ends after the one before it, whether or not it used its results
  if (threadIdx.x == 0) griddep_wait();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while another may still read its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, BN);
  }
}

// ---------------------------------------------------------------- dX

// dX[M x K] by pairs of CTAs (cta_group::2), in tiles of 256 tokens x 256 HALVES columns: a CTA
// loads its 128 tokens of dY and its half of the columns of W per step of 64, the first CTA
// issues the MMAs for both, and each keeps its 128 rows of the accumulator in its own TMEM.
// Persistent; the tiles of a last, partial round are split along N.
// * HALVES = 1: 32 KB a step and CTA, half of what a lone CTA would load per flop, but still
//   bound by L2 when the clock is high (a step takes 0.39 us where the MMAs need 512 cycles).
//   Two accumulators, so that the epilogue of a tile overlaps the next one.
// * HALVES = 2: a quarter fewer bytes per flop (48 KB a step of 1024 cycles); one accumulator
//   fills the TMEM, and the epilogue does not overlap.
// Four stages: with six, the pairs run further apart and meet less of each other's operands in
// L2, and under the power cap N = 28672, K = 8192, M = 8192 took 5% longer.  Tiles go in groups
// of about as many tokens as columns: 1.08 GB of DRAM reads at 8192^3, against 2.05 without.
constexpr int kDxStages = 4;
constexpr int kDxMaxParts = 4;
template <int HALVES>
struct GradDx {
  static constexpr int kCols = 256 * HALVES;
  static constexpr int kStage = 16384 * (1 + HALVES);
  static constexpr int kSmemBytes = kDxStages * kStage + 1024 + 256;
};

struct GradDxParams {
  uint16_t* dX;
  float* part;      // [split tiles][parts][2 CTAs][columns of a tile][128 rows]
  uint32_t* count;  // [split tiles][2][4], zero before the launch
  int* status;
  int M, K;
  int chunks;       // N / 64
  int rchunks;      // steps of u A^T: (hi, lo) x ranks / 64, or 0
  int half;         // columns of hi in u
  int mt, kt;       // tiles of 256 tokens, of columns
  int full, splits, units;  // whole tiles; parts of each later tile; units in all
  int group;        // token tiles that go together, column tile by column tile
  int fail;         // failure tests only: the first pair leaves out one copy
};

struct GradDxUnit {
  int st, part, parts, m, k, c0, nc, nr;  // st: index among the split tiles
};
__device__ __forceinline__ GradDxUnit grad_dx_unit(const GradDxParams& p, int u) {
  GradDxUnit w;
  int t;
  const int nsu = p.units - p.full;  // the parts of split tiles come first
  if (u >= nsu) {
    t = u - nsu;
    w.st = w.part = 0;
    w.parts = 1;
  } else {
    w.st = u / p.splits;
    t = p.full + w.st;
    w.part = u % p.splits;
    w.parts = p.splits;
  }
  const int per = p.group * p.kt, g = t / per, r = t - g * per;
  const int rows = min(p.group, p.mt - g * p.group);
  w.m = g * p.group + r % rows;
  w.k = r / rows;
  w.c0 = static_cast<int>(static_cast<long long>(w.part) * p.chunks / w.parts);
  w.nc = static_cast<int>(static_cast<long long>(w.part + 1) * p.chunks / w.parts) - w.c0;
  w.nr = w.part == 0 ? p.rchunks : 0;
  return w;
}

struct GradDxCtrl {
  uint64_t full[kDxStages], empty[kDxStages];
  uint64_t accfull[2], accempty[2], fin;
  uint32_t tmem;
  int abort;
};

template <int HALVES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGradThreads, 1)
    grad_dx_kernel(const __grid_constant__ GradDxParams p, const __grid_constant__ CUtensorMap mdy,
                   const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mu,
                   const __grid_constant__ CUtensorMap ma) {
  using L = GradDx<HALVES>;
  extern __shared__ uint8_t smem_raw[];
  // the same offset in both CTAs: dynamic shared memory starts alike in every CTA
  uint8_t* smem = align_1024(smem_raw);
  GradDxCtrl* ctrl = reinterpret_cast<GradDxCtrl*>(smem + kDxStages * L::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kDxStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->accfull[b], 1);
      mbar_init(&ctrl->accempty[b], 8);  // the epilogue warps of both CTAs
    }
    mbar_init(&ctrl->fin, 1);
    ctrl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&ctrl->tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem;
  volatile int* abort_flag = &ctrl->abort;
  // u, and the dense weight: the u kernel ends after the expansion.  Every thread waits, so
  // that the bounded waits below do not run while kernels ahead do.
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int s = 0, ph = 0;
      long long issued = 0;
      bool ok = true;
      for (int u = pair; u < p.units && ok; u += pairs) {
        const GradDxUnit w = grad_dx_unit(p, u);
        const int row = w.m * 256 + static_cast<int>(rank) * 128;
        const int col = w.k * L::kCols + static_cast<int>(rank) * 128;
        for (int c = 0; c < w.nc + w.nr; ++c) {
          if (!mbar_wait_pair(&ctrl->empty[s], ph ^ 1) || *abort_flag) {
            atomicOr(p.status, DEV_ERR_TIMEOUT);
            *abort_flag = 1;
            ok = false;
            break;
          }
          // both CTAs' copies count on the first CTA's barrier
          if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * L::kStage);
          const uint32_t bar = map_to_rank(smem_u32(&ctrl->full[s]), 0);
          uint8_t* a = smem + s * L::kStage;
          uint8_t* b = a + 16384;
          if (c < w.nc) {
            const int n = (w.c0 + c) * kGradChunk;
            if (!p.fail || blockIdx.x != 1 || issued != 0) tma_load_2d_pair(a, &mdy, n, row, bar);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
              tma_load_2d_pair(b + h * 16384, &mw, col + h * 256, n, bar);
              tma_load_2d_pair(b + h * 16384 + 8192, &mw, col + h * 256 + 64, n, bar);
            }
          } else {
            const int r = (c - w.nc) * kGradChunk;
            tma_load_2d_pair(a, &mu, r, row, bar);
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              tma_load_2d_pair(b + h * 16384, &ma, r >= p.half ? r - p.half : r, col + h * 256, bar);
          }
          ++issued;
          if (++s == kDxStages) s = 0, ph ^= 1;
        }
      }
      if (*abort_flag) {
        // let the copies in flight land before the CTAs can exit: the first CTA's barriers
        // count both CTAs' bytes, and the second CTA stays until the first one is through
        if (rank == 0)
          for (long long i = issued > kDxStages ? issued - kDxStages : 0; i < issued; ++i)
            mbar_drain(&ctrl->full[i % kDxStages], (i / kDxStages) & 1);
        for (int i = 0; i < 100; ++i) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc_w = idesc_bf16(256, 256, 0, 1), idesc_r = idesc_bf16(256, 256, 0, 0);
      int s = 0, ph = 0, t = 0;
      bool ok = true;
      for (int u = pair; u < p.units && ok; u += pairs, ++t) {
        const GradDxUnit w = grad_dx_unit(p, u);
        const int b = HALVES == 1 ? t & 1 : 0;  // accumulator, and its phase
        const uint32_t bp = HALVES == 1 ? (t >> 1) & 1 : t & 1;
        const uint32_t acc = tmem + b * 256;
        if (!mbar_wait_pair(&ctrl->accempty[b], bp ^ 1) || *abort_flag) {
          atomicOr(p.status, DEV_ERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        for (int c = 0; c < w.nc + w.nr; ++c) {
          if (!mbar_wait_pair(&ctrl->full[s], ph) || *abort_flag) {
            atomicOr(p.status, DEV_ERR_TIMEOUT);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + s * L::kStage), b0 = a0 + 16384;
          if (c < w.nc) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int h = 0; h < HALVES; ++h)
                mma_bf16_pair(acc + h * 256, smem_desc_sw128(a0 + 32 * k, 16, 1024),
                              smem_desc_sw128(b0 + h * 16384 + 2048 * k, 8192, 1024), idesc_w, c != 0 || k != 0);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int h = 0; h < HALVES; ++h)
                mma_bf16_pair(acc + h * 256, smem_desc_sw128(a0 + 32 * k, 16, 1024),
                              smem_desc_sw128(b0 + h * 16384 + 32 * k, 16, 1024), idesc_r, 1u);
          }
          mma_commit_pair(&ctrl->empty[s]);
          if (++s == kDxStages) s = 0, ph ^= 1;
        }
        if (ok) mma_commit_pair(&ctrl->accfull[b]);
      }
      mma_commit_pair(&ctrl->fin);
    }
  } else {
    const int q = warp & 3;
    const int row = 32 * q + lane;
    int t = 0;
    for (int u = pair; u < p.units; u += pairs, ++t) {
      const GradDxUnit w = grad_dx_unit(p, u);
      const int b = HALVES == 1 ? t & 1 : 0;
      const uint32_t bp = HALVES == 1 ? (t >> 1) & 1 : t & 1;
      const uint32_t tm = tmem + b * 256 + (static_cast<uint32_t>(32 * q) << 16);
      const bool ok = mbar_wait_pair(&ctrl->accfull[b], bp) && !*abort_flag;
      if (!ok) {
        atomicOr(p.status, DEV_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const size_t m = static_cast<size_t>(w.m) * 256 + rank * 128 + row;
      const int k0 = w.k * L::kCols, kn = min(L::kCols, p.K - k0);
      uint16_t* out = p.dX + m * p.K + k0;
      const bool live = m < static_cast<size_t>(p.M);
      auto store16 = [&](int c, const float (&v)[16]) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          h[e] = *reinterpret_cast<const uint32_t*>(&x);
        }
        if (live) {
          uint4* o = reinterpret_cast<uint4*>(out + c);
          o[0] = make_uint4(h[0], h[1], h[2], h[3]);
          o[1] = make_uint4(h[4], h[5], h[6], h[7]);
        }
      };
      float* parts = p.part + (static_cast<size_t>(w.st) * w.parts * 2 + rank) * L::kCols * 128 + row;
      constexpr size_t kPartStride = 2 * L::kCols * 128;
      for (int c = 0; c < kn; c += 16) {
        uint32_t x[16];
        float v[16];
        tmem_ld16(tm + c, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(x[e]);
        if (w.parts == 1) {
          store16(c, v);
        } else {
          float* dst = parts + w.part * kPartStride + c * 128;
#pragma unroll
          for (int e = 0; e < 16; ++e) __stcg(dst + e * 128, v[e]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&ctrl->accempty[b]), 0));
      if (w.parts > 1) {
        __threadfence();
        __syncwarp();
        uint32_t last = 0;
        if (lane == 0)
          last = atomicAdd(p.count + (w.st * 2 + rank) * 4 + q, 1u) == static_cast<uint32_t>(w.parts - 1);
        if (__shfl_sync(0xffffffffu, last, 0)) {
          __threadfence();
          // an L2 round trip per 16 columns: every part's loads go out before the first sum
          for (int c = 0; c < kn; c += 16) {
            float v[16], x[kDxMaxParts][16];
#pragma unroll
            for (int k = 0; k < kDxMaxParts; ++k)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                x[k][e] = k < w.parts ? __ldcg(parts + k * kPartStride + (c + e) * 128) : 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              v[e] = x[0][e];
#pragma unroll
              for (int k = 1; k < kDxMaxParts; ++k) v[e] += x[k][e];
            }
            store16(c, v);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // the last signal to this CTA's barriers has arrived, and then
  if (warp == 1 && lane == 0 && !mbar_wait_pair(&ctrl->fin, 0)) atomicOr(p.status, DEV_ERR_TIMEOUT);
  __syncwarp();
  cluster_sync_all();  // neither CTA leaves while the other may still signal or read it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace salr
