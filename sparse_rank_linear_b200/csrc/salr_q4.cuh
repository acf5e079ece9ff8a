// salr_q4.cuh - weights held as 4-bit codes with group scales, and the layer on them for
// up to 64 tokens:  Y = X W^T + (X A) B,  W[n, k] = s (q - z), with s (bf16) and z (an
// integer 0 .. 15) shared by each group of 32, 64 or 128 consecutive columns of a row.
//
// Packed layout (made once per weight).  A unit is 16 rows x 256 columns: 2048 bytes of
// codes, in four 512-byte tiles of 64 columns, of which lane L of a warp holds 16 bytes:
// with g = L / 4, t = L % 4, word 0 is row g, columns 8t .. 8t+7, word 1 row g, columns
// 32 + 8t .. +7, words 2 and 3 the same of row g + 8.  Nibble p of a word is column 2p and
// nibble p + 4 column 2p + 1, so that (w >> 4p) & 0x000f000f is a pair of neighbouring
// columns in the two halves of a register.  One 16-byte load per lane then gives the A
// fragments (16 x 16, row-major) of four m16n8k16 products: product i takes pairs 2(i & 1)
// and 2(i & 1) + 1 of word i / 2, and the matching X fragment is registers 2i, 2i + 1 of
// the 16 values that the lane loads from its token's row, two 16-byte loads straight from
// row-major X.  The order of the 64 columns within a tile's products does not matter, as
// long as both operands agree, and columns 0 .. 31 stay in products 0 and 1 (groups of 32).
// Scales lie [row tile][unit][g][group], a pair (row g, row g + 8) a word; zero points the
// same in bytes.  K is padded to whole units with zero scales; X is not read there.
//
// Arithmetic: 0x4300 | q is bf16 128 + q; minus the bf16 128 + z it is q - z, exactly.  The
// products q x are exact in fp32 and accumulate in fp32 over a group, which is then scaled
// in fp32; t = X A and the adapter's product stay in fp32.  Y is rounded once.
//
// Bound: HBM, by the codes (0.5 byte per weight plus scales).  At M = 1 the rebuild costs
// about 1.4 instructions per weight pair, half of the issue slots at the copy rate.  The
// legacy mma.sync products suffice: up to 64 tokens they stay under the memory time, and
// they take the rebuilt weights from registers, without a trip through shared memory.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "sm100.cuh"

namespace salr {

constexpr int kQ4Unit = 256;                      // columns of a unit
constexpr int kQ4UnitBytes = 16 * kQ4Unit / 2;    // its codes
constexpr int kQ4MaxTokens = 64;
constexpr int kQ4Warps = 8;

struct Q4View {
  const uint8_t* codes;     // [N / 16][units][2048]
  const uint32_t* scales;   // [N / 16][units][8][256 / group] pairs
  const uint16_t* zeros;    // the same, byte pairs; NULL: 8 everywhere
  int N, K, units;
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
// t = X A for up to 64 tokens, in fp32: t[m * R + r].  A CTA takes 8 ranks and MT tokens
// over all of K: every thread multiplies rows k = tid, tid + 256, ... of A (16 bytes each)
// and the CTA adds up in a fixed order.
constexpr int kQ4TThreads = 256;
template <int MT>
__global__ void __launch_bounds__(kQ4TThreads)
    q4_t_kernel(const uint16_t* __restrict__ X, const uint16_t* __restrict__ A, int M, int K, int R,
                float* __restrict__ t) {
  griddep_launch_dependents();  // the layer kernel waits for this grid before it reads t
  __shared__ float part[kQ4TThreads / 32][MT * 8];
  const int r0 = blockIdx.x * 8, m0 = blockIdx.y * MT;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 8; ++r) acc[m][r] = 0.f;
#pragma unroll 4
  for (int k = threadIdx.x; k < K; k += kQ4TThreads) {
    const uint4 a = *reinterpret_cast<const uint4*>(A + static_cast<size_t>(k) * R + r0);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    float av[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      av[2 * i] = __uint_as_float(w[i] << 16);
      av[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m0 + m < M) {
        const float x = __uint_as_float(static_cast<uint32_t>(X[static_cast<size_t>(m0 + m) * K + k]) << 16);
#pragma unroll
        for (int r = 0; r < 8; ++r) acc[m][r] = fmaf(x, av[r], acc[m][r]);
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
      if (lane == 0) part[warp][m * 8 + r] = v;
    }
  __syncthreads();
  if (threadIdx.x < MT * 8) {
    const int m = m0 + threadIdx.x / 8;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kQ4TThreads / 32; ++w) v += part[w][threadIdx.x];
    if (m < M) t[static_cast<size_t>(m) * R + r0 + threadIdx.x % 8] = v;
  }
}

// ------------------------------------------------------------------------------------
// The layer for M <= 8 NT tokens.  A CTA takes one row tile of 16; its warps share the
// units of that tile (warp w takes units w, w + 8, ...), each with its whole accumulator
// in registers, and the eight partial sums meet in shared memory in a fixed order, so
// results repeat bit for bit.
template <int NT, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(32 * kQ4Warps)
    q4_linear_kernel(const Q4View w, const uint16_t* __restrict__ X, int M,
                     const float* __restrict__ t, const uint16_t* __restrict__ B, int R,
                     uint16_t* __restrict__ Y) {
  constexpr int NG = kQ4Unit / GROUP;  // groups of a unit
  __shared__ float part[kQ4Warps][NT * 8][17];
  __shared__ __align__(16) uint16_t bs[128][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tl = lane & 3;
  const int tile = blockIdx.x;

  // the adapter's 16 columns of B, while the codes stream
  for (int i = threadIdx.x; i < 2 * R; i += 32 * kQ4Warps)
    cp_async16(&bs[i >> 1][(i & 1) * 8], B + static_cast<size_t>(i >> 1) * w.N + tile * 16 + (i & 1) * 8);
  cp_async_commit();

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;

  for (int u = warp; u < w.units; u += kQ4Warps) {
    const size_t at = static_cast<size_t>(tile) * w.units + u;
    uint4 code[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) code[b] = q4_stream16(w.codes + at * kQ4UnitBytes + b * 512 + lane * 16);
    uint32_t sc[NG], zp[NG];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      sc[i] = __ldg(w.scales + (at * 8 + g) * NG + i);
      zp[i] = ZEROS ? __ldg(w.zeros + (at * 8 + g) * NG + i) : 0u;
    }
    float c[NT][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int k0 = u * kQ4Unit + b * 64;
      if (k0 >= w.K) break;  // the padding of the last unit
      const uint32_t cw[4] = {code[b].x, code[b].y, code[b].z, code[b].w};
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 32 columns: products 2h and 2h + 1
        const int grp = (b * 64 + h * 32) / GROUP;
        const uint32_t lo = ZEROS ? q4_bias(zp[grp], 0) : 0x43084308u;
        const uint32_t hi = ZEROS ? q4_bias(zp[grp], 1) : 0x43084308u;
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int p = 4 * (2 * i + j);
            a[i][2 * j] = q4_sub2(((cw[h] >> p) & 0x000f000fu) | 0x43004300u, lo);
            a[i][2 * j + 1] = q4_sub2(((cw[2 + h] >> p) & 0x000f000fu) | 0x43004300u, hi);
          }
        const bool first = (b * 64 + h * 32) % GROUP == 0;
        const bool end = (b * 64 + h * 32 + 32) % GROUP == 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (n * 8 + g < M)
            x = __ldg(reinterpret_cast<const uint4*>(X + static_cast<size_t>(n * 8 + g) * w.K + k0 + h * 32 + tl * 8));
          if (first) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
          mma_m16n8k16(c[n], a[0][0], a[0][1], a[0][2], a[0][3], x.x, x.y);
          mma_m16n8k16(c[n], a[1][0], a[1][1], a[1][2], a[1][3], x.z, x.w);
          if (end) {
            const float s0 = __uint_as_float(sc[grp] << 16), s1 = __uint_as_float(sc[grp] & 0xffff0000u);
            acc[n][0] = fmaf(s0, c[n][0], acc[n][0]);
            acc[n][1] = fmaf(s0, c[n][1], acc[n][1]);
            acc[n][2] = fmaf(s1, c[n][2], acc[n][2]);
            acc[n][3] = fmaf(s1, c[n][3], acc[n][3]);
          }
        }
      }
    }
  }

  if (R > 0) {
    cp_async_wait_all();
    __syncthreads();
    griddep_wait();  // t
    for (int r = warp; r < R; r += kQ4Warps) {
      const float b0 = __uint_as_float(static_cast<uint32_t>(bs[r][g]) << 16);
      const float b1 = __uint_as_float(static_cast<uint32_t>(bs[r][g + 8]) << 16);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int m = n * 8 + 2 * tl;
        const float t0 = m < M ? __ldcg(t + static_cast<size_t>(m) * R + r) : 0.f;
        const float t1 = m + 1 < M ? __ldcg(t + static_cast<size_t>(m + 1) * R + r) : 0.f;
        acc[n][0] = fmaf(b0, t0, acc[n][0]);
        acc[n][1] = fmaf(b0, t1, acc[n][1]);
        acc[n][2] = fmaf(b1, t0, acc[n][2]);
        acc[n][3] = fmaf(b1, t1, acc[n][3]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    part[warp][n * 8 + 2 * tl][g] = acc[n][0];
    part[warp][n * 8 + 2 * tl + 1][g] = acc[n][1];
    part[warp][n * 8 + 2 * tl][g + 8] = acc[n][2];
    part[warp][n * 8 + 2 * tl + 1][g + 8] = acc[n][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < M * 16; i += 32 * kQ4Warps) {
    const int m = i >> 4, r = i & 15;
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < kQ4Warps; ++x) v += part[x][m][r];
    reinterpret_cast<__nv_bfloat16*>(Y)[static_cast<size_t>(m) * w.N + tile * 16 + r] = __float2bfloat16_rn(v);
  }
}

// ------------------------------------------------------------------------------------
// The dense bf16 weight [N x K] (s (q - z), rounded once), for larger token counts, the
// gradients and salr_decode.  One warp per unit: each lane writes whole 16-byte pieces,
// four neighbouring lanes 64 consecutive bytes.
template <int GROUP, bool ZEROS>
__global__ void __launch_bounds__(256) q4_expand_kernel(const Q4View w, uint16_t* __restrict__ out) {
  constexpr int NG = kQ4Unit / GROUP;
  griddep_launch_dependents();  // a kernel launched to overlap this one waits for it itself
  const int lane = threadIdx.x & 31, g = lane >> 2, tl = lane & 3;
  const long long total = static_cast<long long>(w.N / 16) * w.units;
  const long long step = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  for (long long at = blockIdx.x * static_cast<long long>(blockDim.x >> 5) + (threadIdx.x >> 5);
       at < total; at += step) {
    const long long tile = at / w.units;
    const int u = static_cast<int>(at - tile * w.units);
    uint4 code[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) code[b] = q4_stream16(w.codes + at * kQ4UnitBytes + b * 512 + lane * 16);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int k0 = u * kQ4Unit + b * 64;
      if (k0 >= w.K) break;
      const uint32_t cw[4] = {code[b].x, code[b].y, code[b].z, code[b].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // word i: row half i / 2, columns (i & 1) * 32 + 8 tl ..
        const int h = i & 1, hi = i >> 1, grp = (b * 64 + h * 32) / GROUP;
        const uint32_t s2 = __ldg(w.scales + (at * 8 + g) * NG + grp);
        const float s = __uint_as_float(hi ? s2 & 0xffff0000u : s2 << 16);
        const float z = ZEROS ? static_cast<float>((__ldg(w.zeros + (at * 8 + g) * NG + grp) >> (8 * hi)) & 255u) : 8.f;
        uint32_t o[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float q0 = static_cast<float>((cw[i] >> (4 * p)) & 15u);
          const float q1 = static_cast<float>((cw[i] >> (4 * p + 16)) & 15u);
          const __nv_bfloat162 v = __floats2bfloat162_rn(s * (q0 - z), s * (q1 - z));
          o[p] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(out + (tile * 16 + g + 8 * hi) * static_cast<size_t>(w.K) + k0 + h * 32 + tl * 8) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// ------------------------------------------------------------------------------------
// Packing (offline): row-major codes, scales and zero points into the layout above.  A
// thread makes one word of codes; the first words of a unit also bring its scales.  A zero
// point above 15 is reported.
__global__ void __launch_bounds__(256)
    q4_pack_kernel(const uint32_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                   const uint8_t* __restrict__ zeros, int N, int K, int group, int units,
                   uint32_t* __restrict__ out_codes, uint32_t* __restrict__ out_scales,
                   uint16_t* __restrict__ out_zeros, int* status) {
  const long long total = static_cast<long long>(N / 16) * units * (kQ4UnitBytes / 4);
  const int ng = kQ4Unit / group, groups = K / group;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long at = i / (kQ4UnitBytes / 4);
    const int word = static_cast<int>(i % (kQ4UnitBytes / 4));
    const long long tile = at / units;
    const int u = static_cast<int>(at % units);
    const int b = word / 128, lane = word % 128 / 4, j = word & 3;
    const long long row = tile * 16 + (lane >> 2) + 8 * (j >> 1);
    const int k = u * kQ4Unit + b * 64 + (j & 1) * 32 + (lane & 3) * 8;
    uint32_t v = 0;
    if (k < K) {
      const uint32_t c = codes[(row * K + k) / 8];  // nibble i: column k + i
#pragma unroll
      for (int p = 0; p < 4; ++p)
        v |= ((c >> (8 * p)) & 15u) << (4 * p) | ((c >> (8 * p + 4)) & 15u) << (4 * p + 16);
    }
    out_codes[i] = v;
    if (word < 8 * ng) {  // pair `word` of the unit's scales: g = word / ng
      const int gi = u * ng + word % ng;
      const long long r0 = tile * 16 + word / ng;
      uint32_t s = 0, z = 0;
      if (gi < groups) {
        s = scales[r0 * groups + gi] | static_cast<uint32_t>(scales[(r0 + 8) * groups + gi]) << 16;
        if (zeros) {
          const uint32_t z0 = zeros[r0 * groups + gi], z1 = zeros[(r0 + 8) * groups + gi];
          if (z0 > 15 || z1 > 15) atomicOr(status, DEV_ERR_FORMAT);
          z = z0 | z1 << 8;
        }
      }
      out_scales[at * 8 * ng + word] = s;
      if (zeros) out_zeros[at * 8 * ng + word] = static_cast<uint16_t>(z);
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
  const int units = (K + kQ4Unit - 1) / kQ4Unit;
  const long long total = static_cast<long long>(N) * units;
  for (long long at = blockIdx.x * 8ll + (threadIdx.x >> 5); at < total; at += gridDim.x * 8ll) {
    const long long row = at / units;
    const int k = static_cast<int>(at % units) * kQ4Unit + lane * 8;
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
