// salr_q4.cuh - weights held as 4-bit codes with group scales, and the layer on them for
// up to 64 tokens:  Y = X W^T + (X A) B,  W[n, k] = s (q - z), with s (bf16) and z (an
// integer 0 .. 15) shared by each group of 32, 64 or 128 consecutive columns of a row.
//
// Packed layout (made once per weight).  A row block is 128 rows; a record is a row block's
// 128 columns (64 in the last one, if K is an odd multiple of 64) and lies in one piece, so
// that one bulk copy brings it: codes, then scales, then zero points.
//   codes   for each 64 columns 4096 bytes: 8 row tiles (16 rows) of 512 bytes, of which lane
//           L of a warp holds 16 bytes.  With g = L / 4, t = L % 4, word 0 is row g, columns
//           8t .. 8t+7, word 1 row g, columns 32 + 8t .. +7, words 2 and 3 the same of row
//           g + 8.  Nibble p of a word is column 2p and nibble p + 4 column 2p + 1, so that
//           (w >> 4p) & 0x000f000f is a pair of neighbouring columns in a register's halves.
//   scales  for each group of columns 256 bytes: [row tile][g] pairs (row g, row g + 8).
//   zeros   for each group of columns 128 bytes: the same pairs in bytes.
// One 16-byte load per lane gives the A fragments (16 x 16, row-major) of four m16n8k16
// products: product i takes pairs 2(i & 1) and 2(i & 1) + 1 of word i / 2, and the matching X
// fragment is registers 2(i & 1), 2(i & 1) + 1 of the 16 bytes at columns 32 (i / 2) + 8t of
// the lane's token.  The order of the columns within a product does not matter, as long as
// both operands agree, and a product stays within 32 columns (groups of 32).
//
// Arithmetic: 0x4300 | q is bf16 128 + q; minus the bf16 128 + z it is q - z, exactly.  The
// products q x are exact in fp32 and accumulate in fp32 over a group (64 columns of it, if it
// is longer), which is then scaled in fp32.  t = X A is summed in fp32 and enters the adapter's
// product with 16 bits of significand.  Y is rounded once.
//
// Bound: HBM, by the codes (0.5 byte per weight plus scales), in the limit.  At the copy rate
// an SM has 46 weights to rebuild per cycle; the rebuild is 0.9 instructions per weight on the
// integer pipe (half of the issue rate), at most 73 weights per cycle, and with the products,
// the scaling and the stages' handshake measured 24 at M = 1 on 28672 x 8192 (34 us, 3.9
// TB/s).  Nothing is full there (issue slots 51%, HBM 60%): two warps a scheduler wait for
// stages and fixed latencies.  m16n8k16 takes 8 cycles per scheduler, so from about 20 tokens on
// the products set the floor: 1024 / M weights per cycle; measured half of that (28672 x 8192 at
// M = 64: 98 us).  The legacy products are the choice because they take the rebuilt weights from
// registers and give each group's sum back in registers, where its fp32 scale is one
// multiply-add; in tensor memory, the scale would have to be rounded into the bf16 weights.
// Short calls are bound by latencies (launch, first copy 2 us, sums over a cluster 2 us): 6.0 us
// for 4096 x 4096 at M = 1, its bytes' time being 1.4.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "salr_grad.cuh"  // the cluster wrappers
#include "sm100.cuh"

namespace salr {

constexpr int kQ4MaxTokens = 64;
constexpr int kQ4Cols = 128;        // columns of a record, and of a pipeline stage
constexpr int kQ4Codes = 128 * kQ4Cols / 2;
constexpr int kQ4MaxRecord = kQ4Codes + 4 * 384;

struct Q4View {
  const uint8_t* data;  // the records, row block by row block
  int N, K, group;
  int zeros;            // records hold zero points (else 8 everywhere)
  // bytes of a record of `cols` columns, of a row block, and where stage s of one starts
  __host__ __device__ int record(int cols) const { return 64 * cols + cols / group * (zeros ? 384 : 256); }
  __host__ __device__ long long block_bytes() const {
    return static_cast<long long>(K / kQ4Cols) * record(kQ4Cols) + (K % kQ4Cols ? record(K % kQ4Cols) : 0);
  }
  __host__ __device__ const uint8_t* at(int block, int stage) const {
    return data + block * block_bytes() + static_cast<long long>(stage) * record(kQ4Cols);
  }
};

__device__ __forceinline__ uint32_t q4_sub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (w & 0x000f000f) | 0x43004300 in one instruction: the constants come in registers (given
// as literals, the compiler spends one instruction on each).
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, uint32_t mask, uint32_t one28) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(one28));
  return d;
}
// A constant the compiler cannot see through.
__device__ __forceinline__ uint32_t q4_opaque(uint32_t c) {
  uint32_t d;
  asm volatile("mov.u32 %0, %1;" : "=r"(d) : "r"(c));
  return d;
}
// (128 + z) twice, from byte `hi` of a pair of zero points
__device__ __forceinline__ uint32_t q4_bias(uint32_t pair, int hi) {
  return 0x43004300u | (((pair >> (8 * hi)) & 255u) * 0x00010001u);
}

// d = a b + c over 16 x 8 x 16; without c, d = a b.
__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_m16n8k16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The A fragments of the two products over 32 reduction steps, for 16 columns of an operand
// that lies with its reduction index as row (64 columns, 128 bytes, to a row, 128-byte
// swizzle; 16-byte chunk `col8` of the 64 columns and the next): ldmatrix turns 8 x 8
// blocks, and its row addresses put the steps in the order of the X fragments.
__device__ __forceinline__ void q4_turned(uint32_t tile, int step0, int col8, int lane, uint32_t (&a)[2][4]) {
  const int mi = lane >> 3, kr = lane & 7;  // block, and its slot among the steps
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = step0 + 8 * (kr >> 1) + 4 * i + 2 * (mi >> 1) + (kr & 1);
    const uint32_t ad = tile + row * 128 + (((col8 + (mi & 1)) ^ (row & 7)) << 4);
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[i][0]), "=r"(a[i][1]), "=r"(a[i][2]), "=r"(a[i][3])
                 : "r"(ad)
                 : "memory");
  }
}

// The token (of 8) of fragment column g.  Neighbouring columns are four rows of X apart, whose
// 16-byte chunks the 128-byte swizzle puts into different halves of the banks.
__device__ __forceinline__ int q4_token(int g) { return (g >> 1) | ((g & 1) << 2); }

// 16 bytes that are read once, past L1.
__device__ __forceinline__ uint4 q4_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Tiled 3-D tensor copy global -> shared (c0 in elements, a multiple of 16 bytes).
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int32_t c0, int32_t c1,
                                            int32_t c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------------------------
// t = X A for up to 8 NT tokens, by one cluster of CTAs, each a part of K: stages of 128
// columns of X and 128 rows of A (all ranks) by TMA, A read transposed (ldmatrix), a row tile
// of 16 ranks a warp.  The fp32 sums meet in shared memory over the cluster, in order, and
// are stored as two bf16 parts, hi = bf16(t) and lo = bf16(t - hi) (16 bits of significand):
// t2[m][64 (r / 32) + r % 32] = hi, lo 32 further on.  Ranks past R are zero.
//
// One small cluster, so that the layer kernel beside it, which needs t at its end only, has
// the machine: 128 ranks x 11008 columns are 2.8 MB, about 3 us for 8 SMs.
constexpr int kQ4TParts = 8;
constexpr int kQ4TWarps = 8;
template <int NT>
struct Q4TLayout {
  static constexpr int kThreads = 32 * (kQ4TWarps + 1);
  static constexpr int kStage = 32768 + NT * 2048;
  static constexpr int kStages = NT <= 4 ? 4 : 3;  // about 130 KB in flight
  static constexpr int kSmemBytes = kStages * kStage + 1024 + 256;
  static constexpr int kSumRow = 132;  // floats: 128 ranks and a pad
  static_assert(kStages * kStage >= NT * 8 * kSumRow * 4, "the stages hold the sums at the end");
};

struct Q4Ctrl {
  uint64_t full[8], empty[8];
  int abort;
};

__device__ __forceinline__ void q4_abort(int* status, Q4Ctrl* c) {
  atomicOr(status, DEV_ERR_TIMEOUT);
  *reinterpret_cast<volatile int*>(&c->abort) = 1;
}
__device__ __forceinline__ bool q4_aborted(Q4Ctrl* c) { return *reinterpret_cast<volatile int*>(&c->abort) != 0; }

template <int NT>
__global__ void __launch_bounds__(Q4TLayout<NT>::kThreads)
    q4_t_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap ma, int M,
                int K, int R, uint16_t* __restrict__ t2, int* status) {
  using L = Q4TLayout<NT>;
  extern __shared__ uint8_t smem_raw[];
  // the same offset in every CTA: dynamic shared memory starts alike in all of them
  uint8_t* smem = align_1024(smem_raw);
  Q4Ctrl* ctrl = reinterpret_cast<Q4Ctrl*>(smem + L::kStages * L::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tl = lane & 3;
  const int part = blockIdx.x, chunks = (K + 127) / 128;
  const int c0 = part * chunks / kQ4TParts, c1 = (part + 1) * chunks / kQ4TParts;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], kQ4TWarps);
    }
    ctrl->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  // X is complete from here on, for the layer kernel too, which this lets start: it waits for
  // this grid before it reads t
  griddep_wait();
  griddep_launch_dependents();
  if (warp == kQ4TWarps) {
    if (lane == 0) {
      int s = 0, ph = 0, issued = 0;
      for (int c = c0; c < c1; ++c) {
        if (!mbar_wait(&ctrl->empty[s], ph ^ 1) || q4_aborted(ctrl)) {
          q4_abort(status, ctrl);
          break;
        }
        uint8_t* a = smem + s * L::kStage;
        uint64_t* bar = &ctrl->full[s];
        // past K, both read as zero
        mbar_arrive_expect_tx(bar, (R > 64 ? 32768 : 16384) + NT * 2048);
        tma_load_2d(a, &ma, 0, c * 128, bar);
        if (R > 64) tma_load_2d(a + 16384, &ma, 64, c * 128, bar);
        tma_load_3d(a + 32768, &mx, 0, 0, 2 * c, bar);
        ++issued;
        if (++s == L::kStages) s = 0, ph ^= 1;
      }
      if (q4_aborted(ctrl))  // let the copies in flight land before the CTA can exit
        for (int i = issued > L::kStages ? issued - L::kStages : 0; i < issued; ++i)
          mbar_drain(&ctrl->full[i % L::kStages], (i / L::kStages) & 1);
    }
  } else {
    const bool live = warp * 16 < R;
    const int tk = q4_token(g);
    int s = 0, ph = 0;
    for (int c = c0; c < c1; ++c) {
      const bool ok = mbar_wait(&ctrl->full[s], ph);
      if (!ok) q4_abort(status, ctrl);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t* tile = smem + s * L::kStage;
      if (live) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t a[2][4];
          q4_turned(smem_u32(tile) + (warp >> 2) * 16384, 32 * h, (warp & 3) * 2, lane, a);
          const uint8_t* x = tile + 32768 + (h >> 1) * NT * 1024 + tk * 128 + (((4 * (h & 1) + tl) ^ tk) << 4);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 v = *reinterpret_cast<const uint4*>(x + n * 1024);
            mma_m16n8k16(acc[n], a[0], v.x, v.y);
            mma_m16n8k16(acc[n], a[1], v.z, v.w);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->empty[s]);
      if (++s == L::kStages) s = 0, ph ^= 1;
    }
  }
  __syncthreads();  // every stage has been used
  float* sums = reinterpret_cast<float*>(smem);  // [8 NT tokens][132]
  if (warp < kQ4TWarps) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float* d = sums + (8 * n + tl) * L::kSumRow + warp * 16 + g;  // tokens tl and tl + 4
      d[0] = acc[n][0];
      d[4 * L::kSumRow] = acc[n][1];
      d[8] = acc[n][2];
      d[4 * L::kSumRow + 8] = acc[n][3];
    }
  }
  __syncthreads();
  cluster_sync_all();
  if (!q4_aborted(ctrl)) {
    // this CTA's 16 ranks of every token
    for (int i = threadIdx.x; i < M * 16; i += L::kThreads) {
      const int m = i / 16, r = part * 16 + i % 16;
      const uint32_t at = smem_u32(sums + m * L::kSumRow + r);
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kQ4TParts; ++k) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(map_to_rank(at, k)));
        v += x;
      }
      if (r >= R) v = 0.f;
      const __nv_bfloat16 hi = __float2bfloat16_rn(v);
      const float h = __bfloat162float(hi);
      // an infinite value is all in hi
      const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(h) <= 3.402823466e38f ? v - h : 0.f);
      uint16_t* o = t2 + m * 256 + r / 32 * 64 + r % 32;
      o[0] = *reinterpret_cast<const uint16_t*>(&hi);
      o[32] = *reinterpret_cast<const uint16_t*>(&lo);
    }
  }
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while another may still read its sums
}

// ------------------------------------------------------------------------------------
// The layer for M <= 8 NT tokens.  Persistent CTAs, several to an SM: the weight's records,
// row block by row block, are cut into one equal contiguous range per CTA, so that every SM
// has the same work whatever the shape.  One producer thread brings each stage (a record or
// two) by one bulk copy and its X tiles by one TMA copy (128-byte swizzle; tokens past M
// read as zero) into a ring; 8 / RT consumer warps, RT row tiles each, rebuild the codes in
// registers and multiply.  The CTA whose range holds a row block's first record also takes
// the block's adapter, after its weight stages: 32 ranks a stage, B by TMA, read
// transposed, t in its two parts.  A block that lies in one range is written at once;
// otherwise the fp32 sums are stored, and q4_sum_kernel adds them up in the order of the
// ranges: results repeat bit for bit.
//
// RT = 2: a warp reads every X fragment once for two row tiles.  With one (twice the warps),
// up_proj M = 24 took 21.5 against 20.4 us, large M = 16 48.0 against 45.5, and one token 1 to
// 2% more.  Deep rings count for more than warps: at one token, three CTAs an SM of three
// stages took 46.3 us on 28672 x 8192 where two of four stages took 37.2.  (All of these with
// the ranges' sums added by the last warp to arrive: q4_sum_kernel brought 28672 x 8192 to 34 us
// at M = 1, 40 at M = 16 with adapters, and from 121 to 98 at M = 64.)
template <int NT>
struct Q4Layout {
  static constexpr int RT = 2;
  static constexpr int kWarps = 8 / RT;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kXHalf = NT * 1024;  // 8 NT tokens x 64 columns
  // Records to a stage: with few tokens a record is so little work that the stage's
  // handshake would take a third of the instructions.
  static constexpr int kRecords = NT <= 4 ? 2 : 1;
  static constexpr int kXBytes = 2 * kRecords * kXHalf;
  static constexpr int kStage = kXBytes + (kRecords * kQ4MaxRecord + 1023) / 1024 * 1024;
  static constexpr int kStages = NT == 4 ? 3 : 4;
  static constexpr int kSmemBytes = kStages * kStage + 1024 + 256;
  static_assert(kStages * kStage >= NT * 8 * 132 * 4, "the stages hold the sums at the end");
  // CTAs per SM that the shared memory admits (1 KB of it is the system's, per CTA)
  static constexpr int kPerSm = 233472 / (kSmemBytes + 1024) > 4 ? 4 : 233472 / (kSmemBytes + 1024);
};

constexpr int kQ4SumRow = 132;  // floats: 128 rows and a pad

struct Q4Params {
  Q4View w;
  uint16_t* Y;
  float* part;      // [2 CTAs][M][128]: a CTA's range has at most two blocks it shares
  int* status;
  int M, R;
  int fail;         // failure tests only: the first CTA leaves out one copy of X
  int parts;        // > 1: clusters of so many CTAs share a row block, one part of its records each
  int records;      // of a row block
  long long total;  // records in all
};

// First record of CTA c's range, of `ctas`; and the CTA whose range holds record i.
__device__ __forceinline__ long long q4_range(long long total, int c, int ctas) { return total * c / ctas; }
__device__ __forceinline__ int q4_owner(long long total, long long i, int ctas) {
  return static_cast<int>(((i + 1) * ctas - 1) / total);
}

// A record of COLS columns into the sums.
template <int NT, int GROUP, bool ZEROS, int COLS>
__device__ __forceinline__ void q4_record(const uint8_t* x, const uint8_t* rec, int warp, int lane,
                                         uint32_t mask, uint32_t one28, uint32_t eight,
                                         float (&acc)[Q4Layout<NT>::RT][NT][4]) {
  using L = Q4Layout<NT>;
  constexpr int RT = L::RT;
  const int g = lane >> 2, tl = lane & 3;
  const uint8_t* codes = rec + warp * (RT * 512) + lane * 16;
  const uint8_t* scales = rec + 64 * COLS + (warp * RT * 8 + g) * 4;
  const uint8_t* zeros = rec + 64 * COLS + COLS / GROUP * 256 + (warp * RT * 8 + g) * 2;
  // this lane's token of each 8, 16-byte chunks tl and 4 + tl of its 64 columns, swizzled
  const int tk = q4_token(g);
  const uint8_t* const xh[2] = {x + tk * 128 + ((tl ^ tk) << 4), x + tk * 128 + (((4 + tl) ^ tk) << 4)};
  // tokens taken at once (of 8 each): their products do not wait for one another, and the
  // fragments of all NT would not fit the registers
  constexpr int NC = NT < 2 ? NT : 2;
#pragma unroll
  for (int b = 0; b < COLS / 64; ++b) {
    uint32_t a[RT][2][2][4];  // [row tile][32 columns][product]
    float sl[RT][2], sh[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint4 code = *reinterpret_cast<const uint4*>(codes + b * 4096 + r * 512);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int grp = (b * 64 + h * 32) / GROUP;
        uint32_t lo = eight, hi = eight;
        if (ZEROS) {
          const uint32_t z = *reinterpret_cast<const uint16_t*>(zeros + grp * 128 + r * 16);
          lo = q4_bias(z, 0);
          hi = q4_bias(z, 1);
        }
        const uint32_t w0 = h ? code.y : code.x, w1 = h ? code.w : code.z;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int at = 4 * (2 * i + j);
            a[r][h][i][2 * j] = q4_sub2(q4_pair(w0 >> at, mask, one28), lo);
            a[r][h][i][2 * j + 1] = q4_sub2(q4_pair(w1 >> at, mask, one28), hi);
          }
        const uint32_t s2 = *reinterpret_cast<const uint32_t*>(scales + grp * 256 + r * 32);
        sl[r][h] = __uint_as_float(s2 << 16);
        sh[r][h] = __uint_as_float(s2 & 0xffff0000u);
      }
    }
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += NC) {
      float cc[RT][NC][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 v[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) v[n] = *reinterpret_cast<const uint4*>(xh[h] + b * L::kXHalf + (n0 + n) * 1024);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            if (h == 0 || GROUP == 32)
              mma_m16n8k16_zero(cc[r][n], a[r][h][0], v[n].x, v[n].y);
            else
              mma_m16n8k16(cc[r][n], a[r][h][0], v[n].x, v[n].y);
          }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int n = 0; n < NC; ++n) mma_m16n8k16(cc[r][n], a[r][h][1], v[n].z, v[n].w);
        if (h == 1 || GROUP == 32) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              float(&d)[4] = acc[r][n0 + n];
              d[0] = fmaf(sl[r][h], cc[r][n][0], d[0]);
              d[1] = fmaf(sl[r][h], cc[r][n][1], d[1]);
              d[2] = fmaf(sh[r][h], cc[r][n][2], d[2]);
              d[3] = fmaf(sh[r][h], cc[r][n][3], d[3]);
            }
        }
      }
    }
  }
}

// A consumer warp: its row tiles of every segment of the CTA's range.
template <int NT, int GROUP, bool ZEROS>
__device__ __forceinline__ void q4_consume(const Q4Params& p, uint8_t* smem, Q4Ctrl* ctrl, long long i0, long long i1,
                                           int ranks, int warp, int lane) {
  using L = Q4Layout<NT>;
  constexpr int RT = L::RT;
  constexpr int kRecord = 64 * kQ4Cols + kQ4Cols / GROUP * (ZEROS ? 384 : 256);  // bytes
  const int cta = blockIdx.x;
  const int g = lane >> 2, tl = lane & 3, tk = q4_token(g);
  // X comes after the kernel ahead: the bounded waits below do not run while that one does
  if (p.R == 0) griddep_wait();
  const uint32_t mask = q4_opaque(0x000f000fu), one28 = q4_opaque(0x43004300u), eight = q4_opaque(0x43084308u);
  int s = 0, ph = 0;
  for (long long i = i0; i < i1;) {
    const int block = static_cast<int>(i / p.records), c0 = static_cast<int>(i - static_cast<long long>(block) * p.records);
    const int n = static_cast<int>(min(static_cast<long long>(p.records - c0), i1 - i));
    const int stages = (n + L::kRecords - 1) / L::kRecords, extra = c0 == 0 ? ranks : 0;
    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int k = 0; k < NT; ++k) acc[r][k][0] = acc[r][k][1] = acc[r][k][2] = acc[r][k][3] = 0.f;
    // records of 128 columns yet to come in this segment; a shorter one ends the block
    int wide = c0 + n == p.records && p.w.K % kQ4Cols ? n - 1 : n;
    const bool narrow = wide < n;
    for (int c = 0; c < stages + extra; ++c) {
      const bool ok = mbar_wait(&ctrl->full[s], ph);
      if (!__all_sync(0xffffffffu, ok)) {
        q4_abort(p.status, ctrl);
        break;
      }
      const uint8_t* x = smem + s * L::kStage;
      const uint8_t* rec = x + L::kXBytes;
      if (c < stages) {
#pragma unroll
        for (int k = 0; k < L::kRecords; ++k, --wide) {
          if (wide > 0)
            q4_record<NT, GROUP, ZEROS, kQ4Cols>(x + k * 2 * L::kXHalf, rec + k * kRecord, warp, lane, mask, one28,
                                                 eight, acc);
          else if (GROUP < 128 && narrow && wide == 0)
            q4_record<NT, GROUP, ZEROS, GROUP == 128 ? 128 : 64>(x + k * 2 * L::kXHalf, rec + k * kRecord, warp,
                                                                 lane, mask, one28, eight, acc);
        }
      } else {
        uint32_t a[RT][2][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int row = (warp * RT + r) * 16;
          q4_turned(smem_u32(rec) + (row >> 6) * 4096, 0, (row & 63) >> 3, lane, a[r]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)  // t's two parts
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            const uint4 v = *reinterpret_cast<const uint4*>(x + k * 1024 + tk * 128 + (((4 * h + tl) ^ tk) << 4));
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              mma_m16n8k16(acc[r][k], a[r][0], v.x, v.y);
              mma_m16n8k16(acc[r][k], a[r][1], v.z, v.w);
            }
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->empty[s]);
      if (++s == L::kStages) s = 0, ph ^= 1;
    }
    if (p.parts > 1) {  // the CTAs of the cluster add them up together
      named_bar(1, 32 * L::kWarps);  // every consumer is through with the ring
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          float* d = reinterpret_cast<float*>(smem) + (8 * k + tl) * kQ4SumRow + (warp * RT + r) * 16 + g;
          d[0] = acc[r][k][0];
          d[4 * kQ4SumRow] = acc[r][k][1];
          d[8] = acc[r][k][2];
          d[4 * kQ4SumRow + 8] = acc[r][k][3];
        }
      return;
    }
    if (q4_aborted(ctrl)) return;  // the values are not whole: nothing of the block is written
    // this warp's rows of the block: values (row, token) at 4 places of each 16 x 8 tile
    const size_t n0 = static_cast<size_t>(block) * 128;
    auto each = [&](auto&& f) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = 8 * k + tl + 4 * (e & 1), row = (warp * RT + r) * 16 + g + 8 * (e >> 1);
            if (m < p.M) f(acc[r][k][e], m, row);
          }
    };
    auto store = [&](float v, int m, int row) {
      reinterpret_cast<__nv_bfloat16*>(p.Y)[static_cast<size_t>(m) * p.w.N + n0 + row] = __float2bfloat16_rn(v);
    };
    if (n == p.records) {
      each(store);
    } else {
      // a block that the range starts in takes the CTA's slot 0, one that it ends in slot 1
      float* mine = p.part + (2 * static_cast<size_t>(cta) + (i == i0 ? 0 : 1)) * (static_cast<size_t>(p.M) * 128);
      each([&](float v, int m, int row) { __stcg(mine + m * 128 + row, v); });
    }
    i += n;
  }
}

// The sums of a cluster's CTAs, which lie in their shared memory ([token][132]): each CTA adds
// up and writes its share of the row block's values, in the order of the parts.
template <int NT>
__device__ __forceinline__ void q4_join(const Q4Params& p, uint8_t* smem, Q4Ctrl* ctrl, int block) {
  const int part = blockIdx.x % p.parts;
  __syncthreads();
  cluster_sync_all();
  if (!q4_aborted(ctrl)) {
    const int all = p.M * 64;  // pairs of rows
    const uint32_t base = smem_u32(smem);
    for (int i = part * all / p.parts + threadIdx.x; i < (part + 1) * all / p.parts; i += Q4Layout<NT>::kThreads) {
      const int m = i >> 6, row = 2 * (i & 63);
      const uint32_t at = base + (m * kQ4SumRow + row) * 4;
      float x[8][2], v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k][0] = x[k][1] = 0.f;
        if (k < p.parts)
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                       : "=f"(x[k][0]), "=f"(x[k][1])
                       : "r"(map_to_rank(at, k)));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v0 += x[k][0], v1 += x[k][1];
      *reinterpret_cast<__nv_bfloat162*>(p.Y + static_cast<size_t>(m) * p.w.N + block * 128 + row) =
          __floats2bfloat162_rn(v0, v1);
    }
  }
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while another may still read its sums
}

template <int NT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(Q4Layout<NT>::kThreads, Q4Layout<NT>::kPerSm)
    q4_linear_kernel(const __grid_constant__ Q4Params p, const __grid_constant__ CUtensorMap mx,
                     const __grid_constant__ CUtensorMap mt, const __grid_constant__ CUtensorMap mb) {
  using L = Q4Layout<NT>;
  constexpr int kRecord = 64 * kQ4Cols + kQ4Cols / GROUP * (ZEROS ? 384 : 256);  // bytes
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1024(smem_raw);
  Q4Ctrl* ctrl = reinterpret_cast<Q4Ctrl*>(smem + L::kStages * L::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const long long i0 = q4_range(p.total, cta, ctas), i1 = q4_range(p.total, cta + 1, ctas);
  const int ranks = (p.R + 31) / 32;  // adapter stages of a block
  griddep_launch_dependents();  // a kernel launched to overlap this one waits for it itself

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], L::kWarps);
    }
    ctrl->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == L::kWarps) {
    if (lane == 0) {
      // a range's records lie one behind another: no addresses are computed per stage (their
      // divisions and 64-bit products took this one thread longer than a stage's products)
      const int first = static_cast<int>(i0 / p.records);
      const uint8_t* rec = p.w.at(first, static_cast<int>(i0 - static_cast<long long>(first) * p.records));
      const uint32_t tail = p.w.K % kQ4Cols ? p.w.record(p.w.K % kQ4Cols) : kRecord;
      // The codes may come before the kernel ahead has completed; X (without adapters: after
      // the t kernel has started, X is complete) and all that is written come after it.
      const bool early = p.R == 0;
      int s = 0, ph = 0, issued = 0;
      bool ok = true, waited = false;
      for (long long i = i0; i < i1 && ok;) {
        const int block = static_cast<int>(i / p.records), c0 = static_cast<int>(i - static_cast<long long>(block) * p.records);
        const int n = static_cast<int>(min(static_cast<long long>(p.records - c0), i1 - i));
        const int stages = (n + L::kRecords - 1) / L::kRecords, extra = c0 == 0 ? ranks : 0;
        const int ahead = early && i == i0 ? min(stages, L::kStages) : 0;
        for (int c = 0; c < stages + extra; ++c) {
          if (!mbar_wait(&ctrl->empty[s], ph ^ 1) || q4_aborted(ctrl)) {
            q4_abort(p.status, ctrl);
            ok = false;
            break;
          }
          uint8_t* x = smem + s * L::kStage;
          uint8_t* dst = x + L::kXBytes;
          uint64_t* bar = &ctrl->full[s];
          if (c < stages) {
            const int at = c0 + c * L::kRecords, cnt = min(L::kRecords, c0 + n - at);
            // the last record of a block may be the shorter one
            const uint32_t bytes = (cnt - 1) * kRecord + (at + cnt == p.records ? tail : kRecord);
            mbar_arrive_expect_tx(bar, bytes + L::kXBytes);
            bulk_g2s(dst, rec, bytes, bar);
            if (c >= ahead && (!p.fail || cta != 0 || issued != 0)) tma_load_3d(x, &mx, 0, 0, 2 * at, bar);
            rec += bytes;
            if (c + 1 == ahead) {  // every stage of the ring has its codes coming
              griddep_wait();
              for (int k = p.fail && cta == 0 ? 1 : 0; k < ahead; ++k)
                tma_load_3d(smem + k * L::kStage, &mx, 0, 0, 2 * (c0 + k * L::kRecords), &ctrl->full[k]);
            }
          } else {
            const int a = c - stages;
            mbar_arrive_expect_tx(bar, 8192 + L::kXHalf);
            tma_load_2d(dst, &mb, block * 128, a * 32, bar);
            tma_load_2d(dst + 4096, &mb, block * 128 + 64, a * 32, bar);
            if (!waited) griddep_wait();  // t
            waited = true;
            tma_load_2d(x, &mt, a * 64, 0, bar);
          }
          ++issued;
          if (++s == L::kStages) s = 0, ph ^= 1;
        }
        i += n;
      }
      if (q4_aborted(ctrl))  // let the copies in flight land before the CTA can exit
        for (int k = issued > L::kStages ? issued - L::kStages : 0; k < issued; ++k)
          mbar_drain(&ctrl->full[k % L::kStages], (k / L::kStages) & 1);
      if (p.R > 0 && !waited) griddep_wait();  // this grid ends after the t kernel
    }
  } else {
    q4_consume<NT, GROUP, ZEROS>(p, smem, ctrl, i0, i1, ranks, warp, lane);
  }
  if (p.parts > 1) q4_join<NT>(p, smem, ctrl, static_cast<int>(i0 / p.records));
}

// The sums of the row blocks that lie in several ranges, added up in the order of the ranges,
// into Y: CTA x takes block x, a warp a token, a lane 4 rows.  A launch of its own, which
// starts with the layer kernel and waits for it: nothing is counted or reset, so the calls on
// a weight share no state.
struct Q4SumParams {
  const float* part;  // as in Q4Params
  uint16_t* Y;
  int M, N, records, ctas;
  long long total;
};
constexpr int kQ4SumWarps = 4;

__global__ void __launch_bounds__(32 * kQ4SumWarps) q4_sum_kernel(const __grid_constant__ Q4SumParams p) {
  griddep_launch_dependents();  // a kernel launched to overlap this one waits for it itself
  const int block = blockIdx.x, m = blockIdx.y * kQ4SumWarps + (threadIdx.x >> 5), row = (threadIdx.x & 31) * 4;
  const long long b0 = static_cast<long long>(block) * p.records;
  const int f = q4_owner(p.total, b0, p.ctas), l = q4_owner(p.total, b0 + p.records - 1, p.ctas);
  griddep_wait();  // in every CTA: this grid ends after the layer kernel
  if (f == l || m >= p.M) return;
  const size_t slot = static_cast<size_t>(p.M) * 128;
  const float* at = p.part + static_cast<size_t>(m) * 128 + row;
  // the first CTA of the block has it in slot 1 unless its range starts with the block
  float4 v = __ldcg(reinterpret_cast<const float4*>(
      at + (2 * static_cast<size_t>(f) + (q4_range(p.total, f, p.ctas) == b0 ? 0 : 1)) * slot));
#pragma unroll 4
  for (int c = f + 1; c <= l; ++c) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(at + 2 * static_cast<size_t>(c) * slot));
    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p.Y + static_cast<size_t>(m) * p.N + block * 128 + row) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// ------------------------------------------------------------------------------------
// The dense bf16 weight [N x K] (s (q - z), rounded once), for larger token counts, the
// gradients and salr_decode.  s (q - z) has up to 12 bits of significand, a bf16 operand 8: the
// rounding is that of a dense bf16 weight, half a step (2^-8) of each product at most, 0.0014 in
// norm where Y's own rounding is 0.0017.  Kept exactly, as two operands, the weight would take
// the tensor cores twice.  One warp per 16 rows x 64 columns: each lane writes whole
// 16-byte pieces, four neighbouring lanes 64 consecutive bytes.
template <int GROUP, bool ZEROS>
__global__ void __launch_bounds__(256) q4_expand_kernel(const Q4View w, uint16_t* __restrict__ out) {
  griddep_launch_dependents();  // a kernel launched to overlap this one waits for it itself
  const int lane = threadIdx.x & 31, g = lane >> 2, tl = lane & 3, rt = threadIdx.x >> 5;
  const int kb = w.K / 64;
  const long long total = static_cast<long long>(w.N / 128) * kb;
  for (long long at = blockIdx.x; at < total; at += gridDim.x) {  // a CTA: 128 rows x 64 columns
    const int block = static_cast<int>(at / kb), b = static_cast<int>(at % kb);
    const uint8_t* rec = w.at(block, b >> 1);
    const int cols = min(kQ4Cols, w.K - (b >> 1) * kQ4Cols);
    const uint32_t* scales = reinterpret_cast<const uint32_t*>(rec + 64 * cols);
    const uint16_t* zeros = reinterpret_cast<const uint16_t*>(rec + 64 * cols + cols / GROUP * 256);
    const uint4 code = q4_stream16(rec + (b & 1) * 4096 + rt * 512 + lane * 16);
    const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // word i: row half i / 2, columns (i & 1) * 32 + 8 tl ..
      const int h = i & 1, hi = i >> 1, grp = ((b & 1) * 64 + h * 32) / GROUP;
      const int pair = (grp * 8 + rt) * 8 + g;
      const uint32_t s2 = __ldg(scales + pair);
      const float s = __uint_as_float(hi ? s2 & 0xffff0000u : s2 << 16);
      const float z = ZEROS ? static_cast<float>((__ldg(zeros + pair) >> (8 * hi)) & 255u) : 8.f;
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float q0 = static_cast<float>((cw[i] >> (4 * p)) & 15u);
        const float q1 = static_cast<float>((cw[i] >> (4 * p + 16)) & 15u);
        const __nv_bfloat162 v = __floats2bfloat162_rn(s * (q0 - z), s * (q1 - z));
        o[p] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(out + (block * 128ll + rt * 16 + g + 8 * hi) * w.K + b * 64 + h * 32 + tl * 8) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ------------------------------------------------------------------------------------
// Packing (offline): row-major codes, scales and zero points into the records.  A thread
// makes one word of codes; 64 threads of each 64 columns of a row block also bring the
// scales of the groups that start there.  A zero point above 15 is reported.
__global__ void __launch_bounds__(256)
    q4_pack_kernel(const uint32_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                   const uint8_t* __restrict__ zeros, const Q4View w, int* status) {
  const int kb = w.K / 64, groups = w.K / w.group;
  const long long total = static_cast<long long>(w.N / 128) * kb * 1024;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int word = static_cast<int>(i % 1024);
    const int b = static_cast<int>(i / 1024 % kb), block = static_cast<int>(i / 1024 / kb);
    const int cols = min(kQ4Cols, w.K - (b >> 1) * kQ4Cols);
    uint8_t* rec = const_cast<uint8_t*>(w.at(block, b >> 1));
    const int rt = word / 128, lane = word % 128 / 4, j = word & 3;
    const long long row = block * 128ll + rt * 16 + (lane >> 2) + 8 * (j >> 1);
    const int k = b * 64 + (j & 1) * 32 + (lane & 3) * 8;
    const uint32_t c = codes[(row * w.K + k) / 8];  // nibble i: column k + i
    uint32_t v = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      v |= ((c >> (8 * p)) & 15u) << (4 * p) | ((c >> (8 * p + 4)) & 15u) << (4 * p + 16);
    reinterpret_cast<uint32_t*>(rec + (b & 1) * 4096)[word] = v;
    // pair `word` % 64 of group `word` / 64 among those that start in these 64 columns
    const int col = b * 64 + word / 64 * w.group;
    if (col < (b + 1) * 64 && col % w.group == 0) {
      const int pair = word % 64, grp = (col % kQ4Cols) / w.group;
      const long long r0 = block * 128ll + pair / 8 * 16 + pair % 8, at = r0 * groups + col / w.group;
      const long long at8 = at + 8ll * groups;
      const uint32_t s0 = scales[at], s1 = scales[at8];
      // a scale that is not finite is refused: applied to a group's sum, it would not give
      // the infinities and NaN of its single products
      if ((s0 & 0x7f80u) == 0x7f80u || (s1 & 0x7f80u) == 0x7f80u) atomicOr(status, DEV_ERR_FORMAT);
      reinterpret_cast<uint32_t*>(rec + 64 * cols)[grp * 64 + pair] = s0 | s1 << 16;
      if (zeros) {
        const uint32_t z0 = zeros[at], z1 = zeros[at8];
        if (z0 > 15 || z1 > 15) atomicOr(status, DEV_ERR_FORMAT);
        reinterpret_cast<uint16_t*>(rec + 64 * cols + cols / w.group * 256)[grp * 64 + pair] =
            static_cast<uint16_t>(z0 | z1 << 8);
      }
    }
  }
}

// Round-to-nearest codes of a bf16 weight (offline), row-major as salr_q4_pack takes them.
// A warp takes 256 consecutive columns of a row, 8 a lane; group / 8 neighbouring lanes
// share a group.  Values that are not finite are reported.
__global__ void __launch_bounds__(256)
    q4_quantise_kernel(const uint16_t* __restrict__ W, int N, int K, int group, int symmetric,
                       uint32_t* __restrict__ codes, uint16_t* __restrict__ scales,
                       uint8_t* __restrict__ zeros, int* status) {
  const int lane = threadIdx.x & 31, span = group / 8;
  const int units = (K + 255) / 256;
  const long long total = static_cast<long long>(N) * units;
  for (long long at = blockIdx.x * 8ll + (threadIdx.x >> 5); at < total; at += gridDim.x * 8ll) {
    const long long row = at / units;
    const int k = static_cast<int>(at % units) * 256 + lane * 8;
    float v[8];
    float lo = 0.f, hi = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = k < K ? __uint_as_float(static_cast<uint32_t>(W[row * K + k + i]) << 16) : 0.f;
      bad |= !(fabsf(v[i]) <= 3.402823466e38f);
      lo = fminf(lo, v[i]);
      hi = fmaxf(hi, v[i]);
    }
    if (bad) atomicOr(status, DEV_ERR_NAN);
    for (int o = 1; o < span; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const float range = symmetric ? __fdiv_rn(fmaxf(hi, -lo), 7.f) : __fdiv_rn(hi - lo, 15.f);
    const __nv_bfloat16 sb = __float2bfloat16_rn(range);
    const float s = __bfloat162float(sb);
    const float z = symmetric ? 8.f : s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 0.f;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(v[i], s)) + z, 0.f), 15.f) : z;
      c |= static_cast<uint32_t>(q) << (4 * i);
    }
    if (k < K) {
      codes[(row * K + k) / 8] = c;
      if (lane % span == 0) {
        scales[row * (K / group) + k / group] = *reinterpret_cast<const uint16_t*>(&sb);
        if (!symmetric) zeros[row * (K / group) + k / group] = static_cast<uint8_t>(z);
      }
    }
  }
}

}  // namespace salr
