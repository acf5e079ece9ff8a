// salr_adamw.cuh - one AdamW step over many tensors in one launch.
//
// For every element, with t the number of this step and g' = grad_scale g:
//   m <- b1 m + (1 - b1) g'          v <- b2 v + (1 - b2) g'^2
//   p <- (1 - lr wd) p - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Every fp32 operation is rounded on its own (no contraction into fused multiply-adds), so
// that the 8-bit codes below do not depend on how a compiler groups the operations; the
// square root is within 2^-23 and the quotient within 2 units in the last place.
//
// 8-bit moments: blocks of 256 consecutive elements of a tensor hold m and r = sqrt(v) as
// e4m3 values x / scale with one fp32 scale = max|x| / 448 per block.  r rather than v: its
// range over a block is half as many binades, and e4m3 has 17 of them (2^-9 .. 448).  A
// positive r never becomes zero (it is held as at least 2^-9 scale): a zero there would
// divide m by eps alone.  A block whose largest magnitude is below 2^-100 is held as zeros
// (448 / max would leave fp32's normal range).  Non-finite values are held as NaN and do
// not enter the block's maximum.
//
// Bound: HBM.  An element moves 28 bytes with bf16 parameters and gradients, fp32 moments
// and master copies, and 10 bytes with 8-bit moments and no master copies, so the work is
// laid out for loads in flight: one warp per 256-element block, 8 elements a thread, the next
// block's loads (up to 96 bytes a thread) issued before this one is worked on.  The tensor
// table travels in the kernel's parameters: no copy, nothing to keep alive, one launch.
// Measured over the 448 adapter tensors (238 M elements) of 32 layers: fp32 moments and master
// copies 1.13 ms, 5.9 TB/s or 0.91 of the measured copy rate; 8-bit moments 0.61 ms, 4.0 TB/s,
// where about 66 instructions an element, at 3 of 4 issue slots, are the bound.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

namespace salr {

constexpr int kAdamBlock = 256;    // elements per warp pass and per 8-bit scale
constexpr int kAdamThreads = 256;  // 8 warps
constexpr float kE4m3Max = 448.f;
constexpr float kE4m3Tiny = 0.001953125f;               // 2^-9, the smallest positive value
constexpr float kAdamFlush = 7.888609052210118e-31f;  // 2^-100

struct AdamTensor {  // as salr_adamw_tensor
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
};

struct AdamScalars {
  double lr, beta1, beta2, weight_decay;
  float eps, b1, ob1, b2, ob2;  // b1 = (float)beta1, ob1 = (float)(1 - beta1), ...
  const float* lr_dev;          // replaces lr when given
  const float* grad_scale;      // NULL: 1
  long long* step;              // [0] steps done, [1] CTAs done (zero between launches)
  int last;                     // this launch ends the step: it advances step[0]
};

// Table of one launch: tensor i covers the 256-element blocks start[i] .. start[i + 1) - 1.
template <int MAXT>
struct AdamTable {
  AdamScalars s;
  int count;
  int start[MAXT + 1];
  AdamTensor t[MAXT];
};

__device__ __forceinline__ double adam_pow(double b, long long t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

// Square roots of 8 values.  The fully rounded instruction sequence branches and takes three
// times as long as this: an approximate reciprocal root and one Newton step, which leaves all
// but few results correctly rounded (8-bit codes next to a border then fall as those of the
// rounded root do).  Values so small or large that the step would leave fp32's range, zero
// among them, take the former.
__device__ __forceinline__ void adam_sqrt8(const float (&v)[8], float (&r)[8]) {
  float low = v[0], high = v[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) low = fminf(low, v[k]), high = fmaxf(high, v[k]);
  if (low >= 1e-30f && high <= 1e37f) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float y;
      asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(v[k]));
      const float s = v[k] * y;
      r[k] = __fmaf_rn(__fmaf_rn(-s, s, v[k]), 0.5f * y, s);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = __fsqrt_rn(v[k]);
  }
}

// 8 values as they lie in memory, loaded ahead of their use.
template <typename T>
struct AdamRaw;
template <>
struct AdamRaw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load(const float* p, int cnt) {  // the first cnt; the rest 0
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < cnt ? p[k] : 0.f;
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <>
struct AdamRaw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int cnt) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + 2 * k;
      w[k] = (2 * k < cnt ? q[0] : 0u) | (2 * k + 1 < cnt ? static_cast<uint32_t>(q[1]) << 16 : 0u);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void adam_store8(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ void adam_store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void adam_set(float* p, float x) { *p = x; }
__device__ __forceinline__ void adam_set(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The `cnt` (0 .. 8) values from p on, by vectors where allowed.
template <typename T>
__device__ __forceinline__ void adam_get(AdamRaw<T>& r, const T* p, int cnt, bool vec) {
  if (vec && cnt == 8)
    r.load(p);
  else
    r.load(p, cnt);
}
template <typename T>
__device__ __forceinline__ void adam_put(T* p, int cnt, bool vec, const float (&x)[8]) {
  if (vec && cnt == 8) {
    adam_store8(p, x);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < cnt) adam_set(p + k, x[k]);
  }
}

// The thread's 8 codes at element i.  Codes start 8-byte aligned in every tensor, and the
// caller pads a tensor's codes to whole blocks.
__device__ __forceinline__ uint2 adam_codes(const void* p, int64_t i) {
  return __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + i));
}
__device__ __forceinline__ void adam_decode(uint2 c, float scale, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = (k < 2 ? c.x : c.y) >> (16 * (k & 1));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * k] = __fmul_rn(f.x, scale);
    x[2 * k + 1] = __fmul_rn(f.y, scale);
  }
}
__device__ __forceinline__ uint32_t adam_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
// The larger value, or NaN if either is.
__device__ __forceinline__ float adam_max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float adam_warp_max_nan(float a) {
  float d;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(a));
  return d;
}
// a / x by an approximate reciprocal, one Newton step for it and one for the quotient, for x
// within 2^-100 .. 1e37.
__device__ __forceinline__ float adam_quotient(float a, float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  y = __fmaf_rn(y, __fmaf_rn(-x, y, 1.f), y);
  const float q = a * y;
  return __fmaf_rn(__fmaf_rn(-x, q, a), y, q);
}

// Store x (8 values a thread, the warp's block) as e4m3 codes at element i and the block's
// scale at *sp.  All 32 lanes call it together.
template <bool POSITIVE>
__device__ __forceinline__ void adam_encode(const float (&x)[8], void* codes, int64_t i, float* sp,
                                            int lane) {
  constexpr float kMax = 3.402823466e38f;
  float top = fabsf(x[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) top = adam_max_nan(top, fabsf(x[k]));
  top = adam_warp_max_nan(top);
  const bool plain = top <= 1e37f;  // the same in every lane
  float inv = adam_quotient(kE4m3Max, top);
  if (!plain) {  // infinite or NaN, of which the largest finite value counts, or near overflow
    top = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (fabsf(x[k]) <= kMax) top = fmaxf(top, fabsf(x[k]));
    top = adam_warp_max_nan(top);
    inv = __fdiv_rn(kE4m3Max, top);
  }
  const bool live = top >= kAdamFlush;
  if (!live) inv = 0.f;
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = __fmul_rn(x[k], inv);
  if (POSITIVE && live) {  // what is above zero stays so
    float low = x[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) low = fminf(low, x[k]);
    if (low > 0.f) {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = fmaxf(y[k], kE4m3Tiny);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = x[k] > 0.f ? fmaxf(y[k], kE4m3Tiny) : y[k];
    }
  }
  if (!plain) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (!(fabsf(x[k]) <= kMax)) y[k] = __int_as_float(0x7fffffff);  // NaN is held as NaN
  }
  __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(codes) + i),
         make_uint2(adam_e4m3x4(y[0], y[1], y[2], y[3]), adam_e4m3x4(y[4], y[5], y[6], y[7])));
  if (lane == 0) *sp = live ? adam_quotient(top, kE4m3Max) : 0.f;
}

template <int MAXT, typename PT, typename GT, bool MASTER, bool EIGHT>
__global__ void __launch_bounds__(kAdamThreads, EIGHT ? 4 : 3)
    salr_adamw_kernel(const __grid_constant__ AdamTable<MAXT> tab) {
  __shared__ float sh[4];
  const int lane = threadIdx.x & 31;
  const int total = tab.start[tab.count];
  long long t = 0;
  if (threadIdx.x == 0) {
    t = tab.s.step[0] + 1;
    const double lr = tab.s.lr_dev ? static_cast<double>(*tab.s.lr_dev) : tab.s.lr;
    sh[0] = static_cast<float>(lr / (1.0 - adam_pow(tab.s.beta1, t)));
    sh[1] = static_cast<float>(1.0 / sqrt(1.0 - adam_pow(tab.s.beta2, t)));
    sh[2] = static_cast<float>(1.0 - lr * tab.s.weight_decay);
    sh[3] = tab.s.grad_scale ? *tab.s.grad_scale : 1.f;
  }
  __syncthreads();
  const float rate = sh[0], root = sh[1], decay = sh[2], gscale = sh[3];
  const float eps = tab.s.eps, b1 = tab.s.b1, ob1 = tab.s.ob1, b2 = tab.s.b2, ob2 = tab.s.ob2;

  // A CTA takes a contiguous range of blocks, so that its warps look a tensor up only where
  // one ends (a search for every block took 7 of some 100 instructions per 8-bit element).
  const int first = static_cast<int>(static_cast<int64_t>(blockIdx.x) * total / gridDim.x);
  const int behind = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * total / gridDim.x);
  // One block of this warp as loaded; the next one's loads go out before it is worked on.
  struct Loaded {
    int tensor;
    int64_t blk;
    AdamRaw<GT> g;
    AdamRaw<typename std::conditional<MASTER, float, PT>::type> p;
    AdamRaw<float> m, v;
    uint2 mc, vc;
    float ms, vs;
  };
  int lo = 0, end = 0;  // the tensor of the block loaded last, and the block behind it
  auto place = [&](const AdamTensor& e, int64_t blk, int64_t& i, int& cnt, bool& vec) {
    i = blk * kAdamBlock + lane * 8;
    const int64_t left = e.n - i;
    cnt = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
    vec = ((reinterpret_cast<uintptr_t>(e.param) | reinterpret_cast<uintptr_t>(e.grad)) & 15) == 0;
  };
  auto load = [&](int b, Loaded& d) {
    if (b >= end) {
      int hi = tab.count;  // start[lo] <= b < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.start[mid] <= b)
          lo = mid;
        else
          hi = mid;
      }
      end = tab.start[lo + 1];
    }
    const AdamTensor& e = tab.t[lo];
    d.tensor = lo;
    d.blk = b - tab.start[lo];
    int64_t i;
    int cnt;
    bool vec;
    place(e, d.blk, i, cnt, vec);
    adam_get(d.g, static_cast<const GT*>(e.grad) + i, cnt, vec);
    if constexpr (MASTER)
      adam_get(d.p, e.master + i, cnt, true);
    else
      adam_get(d.p, static_cast<const PT*>(e.param) + i, cnt, vec);
    if (EIGHT) {
      d.mc = adam_codes(e.m, i);
      d.vc = adam_codes(e.v, i);
      d.ms = e.m_scale[d.blk];
      d.vs = e.v_scale[d.blk];
    } else {
      adam_get(d.m, static_cast<const float*>(e.m) + i, cnt, true);
      adam_get(d.v, static_cast<const float*>(e.v) + i, cnt, true);
    }
  };
  auto work = [&](const Loaded& d) {
    const AdamTensor& e = tab.t[d.tensor];
    int64_t i;
    int cnt;
    bool vec;
    place(e, d.blk, i, cnt, vec);
    float g[8], p[8], m[8], v[8], r[8];
    d.g.get(g);
    d.p.get(p);
    if (EIGHT) {
      adam_decode(d.mc, d.ms, m);
      adam_decode(d.vc, d.vs, v);
    } else {
      d.m.get(m);
      d.v.get(v);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gk = __fmul_rn(g[k], gscale);
      if (EIGHT) v[k] = __fmul_rn(v[k], v[k]);
      m[k] = __fadd_rn(__fmul_rn(m[k], b1), __fmul_rn(gk, ob1));
      v[k] = __fadd_rn(__fmul_rn(v[k], b2), __fmul_rn(__fmul_rn(gk, gk), ob2));
    }
    adam_sqrt8(v, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float step = __fdividef(m[k], __fadd_rn(__fmul_rn(r[k], root), eps));
      p[k] = __fsub_rn(__fmul_rn(p[k], decay), __fmul_rn(rate, step));
    }
    if (EIGHT) {
      if (cnt < 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k >= cnt) m[k] = r[k] = 0.f;  // past the tensor's end (codes there are padding)
      }
      adam_encode<false>(m, e.m, i, e.m_scale + d.blk, lane);
      adam_encode<true>(r, e.v, i, e.v_scale + d.blk, lane);
    } else {
      adam_put(static_cast<float*>(e.m) + i, cnt, true, m);
      adam_put(static_cast<float*>(e.v) + i, cnt, true, v);
    }
    if (MASTER) adam_put(e.master + i, cnt, true, p);
    adam_put(static_cast<PT*>(e.param) + i, cnt, vec, p);
  };
  int b = first + (threadIdx.x >> 5);
  if (b < behind) {
    Loaded now;
    load(b, now);
    for (b += kAdamThreads / 32; b < behind; b += kAdamThreads / 32) {
      Loaded next;
      load(b, next);
      work(now);
      now = next;
    }
    work(now);
  }

  // The last CTA of the step's last launch advances the step count: every CTA has read it
  // by then (thread 0 reads it before it counts itself out).
  if (tab.s.last) {
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long* done = reinterpret_cast<unsigned long long*>(tab.s.step + 1);
      if (atomicAdd(done, 1ull) == gridDim.x - 1) {
        *done = 0;
        tab.s.step[0] = t;
      }
    }
  }
}

}  // namespace salr
