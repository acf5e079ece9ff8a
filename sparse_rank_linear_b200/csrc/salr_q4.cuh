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
// products q x are exact in fp32 and accumulate in fp32 over a group, which is then scaled
// in fp32.  t = X A is summed in fp32 and enters the adapter's product with 16 bits of
// significand.  Y is rounded once.
//
// Bound: HBM, by the codes (0.5 byte per weight plus scales), up to about 20 tokens; above,
// the products: m16n8k16 at 8 cycles per scheduler leaves 1024 / M weights per cycle and SM,
// against 46 at the copy rate.  The rebuild takes 1.4 instructions per weight, half of the
// issue slots at the copy rate.  The legacy products are the choice because they take the
// rebuilt weights from registers and give each group's sum back in registers, where its
// fp32 scale is one multiply-add; in tensor memory, the scale would have to be rounded into
// the bf16 weights.
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
// (128 + z) twice, from byte `hi` of a pair of zero points
__device__ __forceinline__ uint32_t q4_bias(uint32_t pair, int hi) {
  return 0x43004300u | (((pair >> (8 * hi)) & 255u) * 0x00010001u);
}

__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes that are read once, past L1.
__device__ __forceinline__ uint4 q4_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// ------------------------------------------------------------------------------------
// t = X A for up to 64 tokens, summed in fp32 and stored as two bf16 parts, hi = bf16(t) and
// lo = bf16(t - hi) (16 bits of significand): t2[m][64 (r / 32) + r % 32] = hi, lo 32 further
// on; ranks past R up to a multiple of 32 are zero.  A cluster of CTAs takes 8 ranks and MT
// tokens, each CTA a part of K: every thread multiplies rows k of A (16 bytes each), and the
// parts meet in the first CTA's shared memory, all in a fixed order.
constexpr int kQ4TThreads = 256;
template <int MT>
__global__ void __launch_bounds__(kQ4TThreads)
    q4_t_kernel(const uint16_t* __restrict__ X, const uint16_t* __restrict__ A, int M, int K, int R,
                int parts, uint16_t* __restrict__ t2) {
  griddep_launch_dependents();  // the layer kernel waits for this grid before it reads t
  __shared__ float warps[kQ4TThreads / 32][MT * 8];
  __shared__ float sums[8][MT * 8];  // the first CTA's: one row a part
  const int part = blockIdx.x % parts;
  const int r0 = blockIdx.x / parts * 8, m0 = blockIdx.y * MT;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k0 = static_cast<int>(static_cast<long long>(part) * K / parts);
  const int k1 = static_cast<int>(static_cast<long long>(part + 1) * K / parts);
  float acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 8; ++r) acc[m][r] = 0.f;
  if (r0 < R) {
#pragma unroll 2
    for (int k = k0 + threadIdx.x; k < k1; k += kQ4TThreads) {
      const uint4 a = *reinterpret_cast<const uint4*>(A + static_cast<size_t>(k) * R + r0);
      float x[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        x[m] = m0 + m < M ? __uint_as_float(static_cast<uint32_t>(X[static_cast<size_t>(m0 + m) * K + k]) << 16) : 0.f;
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a0 = __uint_as_float(w[i] << 16), a1 = __uint_as_float(w[i] & 0xffff0000u);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[m][2 * i] = fmaf(x[m], a0, acc[m][2 * i]);
          acc[m][2 * i + 1] = fmaf(x[m], a1, acc[m][2 * i + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      float v = acc[m][r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) warps[warp][m * 8 + r] = v;
    }
  __syncthreads();
  cluster_sync_all();  // every CTA of the cluster runs: its shared memory may be written
  if (threadIdx.x < MT * 8) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kQ4TThreads / 32; ++w) v += warps[w][threadIdx.x];
    const uint32_t to = map_to_rank(smem_u32(&sums[part][threadIdx.x]), 0);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
  }
  __syncthreads();
  cluster_sync_all();
  if (part == 0 && threadIdx.x < MT * 8) {
    float v = 0.f;
    for (int k = 0; k < parts; ++k) v += sums[k][threadIdx.x];
    const int m = m0 + threadIdx.x / 8, r = r0 + threadIdx.x % 8;
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    const float h = __bfloat162float(hi);
    // an infinite value is all in hi
    const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(h) <= 3.402823466e38f ? v - h : 0.f);
    if (m < M) {
      uint16_t* o = t2 + m * 256 + r / 32 * 64 + r % 32;
      o[0] = *reinterpret_cast<const uint16_t*>(&hi);
      o[32] = *reinterpret_cast<const uint16_t*>(&lo);
    }
  }
}

// ------------------------------------------------------------------------------------
// The layer for M <= 8 NT tokens.  A cluster of CTAs takes a row block, each CTA a part of
// its stages (128 columns).  One producer thread brings each stage's record by one bulk copy
// and its X tiles by TMA (128-byte swizzle; tokens past M read as zero) into a ring; 8 / RT
// consumer warps, RT row tiles each, rebuild the codes in registers and multiply.  After the
// weight's stages come the adapter's, 32 ranks each: B by TMA, read transposed (ldmatrix), t
// in its two parts from the t kernel.  The CTAs' sums meet in shared memory over the
// cluster, in the order of the parts: results repeat bit for bit.
//
// RT = 2 from 17 tokens on: a warp reads every X fragment once for its row tiles, and at 64
// tokens one row tile a warp would read 16 bytes of X from shared memory per byte of codes.
template <int NT>
struct Q4Layout {
  static constexpr int RT = NT <= 2 ? 1 : 2;
  static constexpr int kWarps = 8 / RT;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kXHalf = NT * 1024;  // 8 NT tokens x 64 columns
  static constexpr int kStage = 2 * kXHalf + 10240;
  static constexpr int kStages = NT == 1 ? 5 : NT == 2 ? 5 : 4;
  static constexpr int kSmemBytes = kStages * kStage + 1024 + 256;
  static constexpr int kSumRow = 132;  // floats: 128 rows and a pad
  static_assert(kQ4MaxRecord <= 10240 && kStages * kStage >= NT * 8 * kSumRow * 4, "stage sizes");
};

struct Q4Ctrl {
  uint64_t full[8], empty[8];
  int abort;
};

struct Q4Params {
  Q4View w;
  uint16_t* Y;
  int* status;
  int M, R;
  int parts;   // CTAs of a cluster
};

__device__ __forceinline__ uint4 q4_lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t q4_lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t q4_lds2(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

template <int NT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(Q4Layout<NT>::kThreads)
    q4_linear_kernel(const __grid_constant__ Q4Params p, const __grid_constant__ CUtensorMap mx,
                     const __grid_constant__ CUtensorMap mt, const __grid_constant__ CUtensorMap mb) {
  using L = Q4Layout<NT>;
  constexpr int RT = L::RT;
  extern __shared__ uint8_t smem_raw[];
  // the same offset in every CTA: dynamic shared memory starts alike in all of them
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Q4Ctrl* ctrl = reinterpret_cast<Q4Ctrl*>(smem + L::kStages * L::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x % p.parts, block = blockIdx.x / p.parts;
  const int stages = (p.w.K + kQ4Cols - 1) / kQ4Cols, ranks = (p.R + 31) / 32;
  const int s0 = static_cast<int>(static_cast<long long>(part) * stages / p.parts);
  const int s1 = static_cast<int>(static_cast<long long>(part + 1) * stages / p.parts);
  // the adapter's stages are shared out as well
  const int a0 = part * ranks / p.parts, a1 = (part + 1) * ranks / p.parts;
  volatile int* abort_flag = &ctrl->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], L::kWarps);
    }
    ctrl->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();

  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.f;

  if (warp == L::kWarps) {
    if (lane == 0) {
      int s = 0, ph = 0, issued = 0;
      for (int c = s0; c < s1 + a1 - a0; ++c) {
        if (!mbar_wait(&ctrl->empty[s], ph ^ 1) || *abort_flag) {
          atomicOr(p.status, DEV_ERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        uint8_t* x = smem + s * L::kStage;
        uint8_t* rec = x + 2 * L::kXHalf;
        uint64_t* bar = &ctrl->full[s];
        if (c < s1) {
          const int cols = min(kQ4Cols, p.w.K - c * kQ4Cols);
          const uint32_t bytes = static_cast<uint32_t>(p.w.record(cols));
          mbar_arrive_expect_tx(bar, bytes + cols / 64 * L::kXHalf);
          bulk_g2s(rec, p.w.at(block, c), bytes, bar);
          tma_load_2d(x, &mx, c * kQ4Cols, 0, bar);
          if (cols > 64) tma_load_2d(x + L::kXHalf, &mx, c * kQ4Cols + 64, 0, bar);
        } else {
          const int a = a0 + c - s1;
          if (c == s1) griddep_wait();  // t
          mbar_arrive_expect_tx(bar, 8192 + L::kXHalf);
          tma_load_2d(rec, &mb, block * 128, a * 32, bar);
          tma_load_2d(rec + 4096, &mb, block * 128 + 64, a * 32, bar);
          tma_load_2d(x, &mt, a * 64, 0, bar);
        }
        ++issued;
        if (++s == L::kStages) s = 0, ph ^= 1;
      }
      if (*abort_flag)  // let the copies in flight land before the CTA can exit
        for (int i = issued > L::kStages ? issued - L::kStages : 0; i < issued; ++i)
          mbar_wait(&ctrl->full[i % L::kStages], (i / L::kStages) & 1);
    }
  } else {
    const int g = lane >> 2, tl = lane & 3;
    // this lane's X addresses within a half: token 8n + g, 16-byte chunk (4 h + tl), swizzled
    const uint32_t xrow = static_cast<uint32_t>(g * 128);
    const uint32_t xc[2] = {xrow + ((static_cast<uint32_t>(tl) ^ g) << 4),
                            xrow + ((static_cast<uint32_t>(4 + tl) ^ g) << 4)};
    int s = 0, ph = 0;
    bool ok = true;
    for (int c = s0; c < s1 + a1 - a0; ++c) {
      ok = mbar_wait(&ctrl->full[s], ph) && !*abort_flag;
      if (!ok) {
        atomicOr(p.status, DEV_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t x = smem_u32(smem + s * L::kStage), rec = x + 2 * L::kXHalf;
      if (c < s1) {
        const int cols = min(kQ4Cols, p.w.K - c * kQ4Cols);
        const uint32_t sc0 = rec + 64 * cols, zp0 = sc0 + cols / GROUP * 256;
        float cc[RT][NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b * 64 >= cols) break;
          uint4 code[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r)
            code[r] = q4_lds16(rec + b * 4096 + (warp * RT + r) * 512 + lane * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 32 columns, two products
            const int grp = (b * 64 + h * 32) / GROUP;
            const bool first = (b * 64 + h * 32) % GROUP == 0;
            const bool end = (b * 64 + h * 32 + 32) % GROUP == 0;
            uint32_t a[RT][2][4];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const uint32_t at = (grp * 8 + warp * RT + r) * 8 + g;
              uint32_t lo = 0x43084308u, hi = 0x43084308u;
              if (ZEROS) {
                const uint32_t z = q4_lds2(zp0 + at * 2);
                lo = q4_bias(z, 0);
                hi = q4_bias(z, 1);
              }
              const uint32_t w0 = h ? code[r].y : code[r].x, w1 = h ? code[r].w : code[r].z;
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const int sh = 4 * (2 * i + j);
                  a[r][i][2 * j] = q4_sub2(((w0 >> sh) & 0x000f000fu) | 0x43004300u, lo);
                  a[r][i][2 * j + 1] = q4_sub2(((w1 >> sh) & 0x000f000fu) | 0x43004300u, hi);
                }
            }
            float sl[RT], sh[RT];
            if (end) {
#pragma unroll
              for (int r = 0; r < RT; ++r) {
                const uint32_t s2 = q4_lds4(sc0 + ((grp * 8 + warp * RT + r) * 8 + g) * 4);
                sl[r] = __uint_as_float(s2 << 16);
                sh[r] = __uint_as_float(s2 & 0xffff0000u);
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 v = q4_lds16(x + b * L::kXHalf + n * 1024 + xc[h]);
#pragma unroll
              for (int r = 0; r < RT; ++r) {
                float(&d)[4] = cc[r][n];
                if (first) d[0] = d[1] = d[2] = d[3] = 0.f;
                mma_m16n8k16(d, a[r][0][0], a[r][0][1], a[r][0][2], a[r][0][3], v.x, v.y);
                mma_m16n8k16(d, a[r][1][0], a[r][1][1], a[r][1][2], a[r][1][3], v.z, v.w);
                if (end) {
                  acc[r][n][0] = fmaf(sl[r], d[0], acc[r][n][0]);
                  acc[r][n][1] = fmaf(sl[r], d[1], acc[r][n][1]);
                  acc[r][n][2] = fmaf(sh[r], d[2], acc[r][n][2]);
                  acc[r][n][3] = fmaf(sh[r], d[3], acc[r][n][3]);
                }
              }
            }
          }
        }
      } else {
        // 32 ranks: B is [rank][64 rows] twice, 128-byte swizzled.  ldmatrix turns 8 ranks x
        // 8 rows; its row addresses put the ranks in the order of the t fragments.
        const int mi = lane >> 3, kr = lane & 7;  // matrix, and its k slot
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a[RT][4];
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int rank = 8 * (kr >> 1) + 4 * i + 2 * (mi >> 1) + (kr & 1);
            const int row = (warp * RT + r) * 16 + 8 * (mi & 1);
            const uint32_t ad = rec + (row >> 6) * 4096 + rank * 128 +
                                ((static_cast<uint32_t>((row & 63) >> 3) ^ (rank & 7)) << 4);
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(a[r][0]), "=r"(a[r][1]), "=r"(a[r][2]), "=r"(a[r][3])
                         : "r"(ad));
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)  // t's two parts
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 v = q4_lds16(x + n * 1024 + xc[h]);
#pragma unroll
              for (int r = 0; r < RT; ++r)
                mma_m16n8k16(acc[r][n], a[r][0], a[r][1], a[r][2], a[r][3], i ? v.z : v.x, i ? v.w : v.y);
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
  if (warp < L::kWarps) {
    const int g = lane >> 2, tl = lane & 3;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float* d = sums + (8 * n + 2 * tl) * L::kSumRow + (warp * RT + r) * 16 + g;
        d[0] = acc[r][n][0];
        d[L::kSumRow] = acc[r][n][1];
        d[8] = acc[r][n][2];
        d[L::kSumRow + 8] = acc[r][n][3];
      }
  }
  __syncthreads();
  if (p.parts > 1) cluster_sync_all();
  if (*abort_flag == 0) {
    const int rows = 128 / p.parts, r0 = part * rows;
    const uint32_t base = smem_u32(sums);
    for (int i = threadIdx.x; i < p.M * (rows / 2); i += L::kThreads) {
      const int m = i / (rows / 2), row = r0 + i % (rows / 2) * 2;
      const uint32_t at = base + (m * L::kSumRow + row) * 4;
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < p.parts) {
          float x0, x1;
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                       : "=f"(x0), "=f"(x1)
                       : "r"(map_to_rank(at, k)));
          v0 += x0;
          v1 += x1;
        }
      *reinterpret_cast<__nv_bfloat162*>(p.Y + static_cast<size_t>(m) * p.w.N + block * 128 + row) =
          __floats2bfloat162_rn(v0, v1);
    }
  }
  if (p.R > 0 && threadIdx.x == 0) griddep_wait();  // this grid ends after the t kernel
  if (p.parts > 1) {
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while another may still read its sums
  }
}

// ------------------------------------------------------------------------------------
// The dense bf16 weight [N x K] (s (q - z), rounded once), for larger token counts, the
// gradients and salr_decode.  One warp per 16 rows x 64 columns: each lane writes whole
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
      reinterpret_cast<uint32_t*>(rec + 64 * cols)[grp * 64 + pair] =
          scales[at] | static_cast<uint32_t>(scales[at8]) << 16;
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
