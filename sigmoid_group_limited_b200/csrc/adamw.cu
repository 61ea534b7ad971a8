// adamw.cu - one AdamW step over many tensors (moe_adamw_step), states in
// fp32 or in 8 bits.
//
// Bound by HBM: 28 bytes per element with fp32 states, a bf16 parameter, its
// master and a bf16 gradient; 10.06 with 8-bit states and no master. One
// launch takes as many tensors as its parameter block holds; the work is the
// list of all tensors' 256-element blocks, a warp per block (8 elements, 16
// bytes of bf16, per lane), so a block's maximum for the 8-bit scales is one
// warp reduction and nothing is read twice. No atomics: an element is owned
// by one lane.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace sgl {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kBlock = MOE_STATE_BLOCK;  // 32 lanes x 8 elements
constexpr int kMaxTensors = 40;          // per launch: 4 KB of kernel parameters

struct AdamTensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  long long n;
  float wd;  // weight decay of this tensor
  int types; // bit 0: p fp32, bit 1: master, bit 2: g fp32, bit 3: 8-bit states
};

struct AdamParams {
  int count;
  float lr, c1, rc2, gs;  // rate, 1 - beta1^t, sqrt(1 - beta2^t), gradient scale
  float b1, b1c, b2, b2c, eps;
  const float* dyn;
  long long first[kMaxTensors + 1];  // prefix sums of the tensors' blocks
  AdamTensor t[kMaxTensors];
};

// Each load and store moves the 8 elements of a lane's piece; of a tensor's
// last block only n of them exist (FULL: all 8).
template <bool FULL>
__device__ __forceinline__ void load_bf16(const void* base, long long at, int n, float* f) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  if (FULL) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r[i] << 16);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = i < n ? __uint_as_float(static_cast<uint32_t>(p[i]) << 16) : 0.f;
  }
}
template <bool FULL>
__device__ __forceinline__ void load_f32(const void* base, long long at, int n, float* f) {
  const float* p = static_cast<const float*>(base) + at;
  if (FULL) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.f;
  }
}
template <bool FULL>
__device__ __forceinline__ void store_bf16(void* base, long long at, int n, const float* f) {
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if (FULL) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(r[0], r[1], r[2], r[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(r[i / 2] >> (16 * (i & 1)));
  }
}
template <bool FULL>
__device__ __forceinline__ void store_f32(void* base, long long at, int n, const float* f) {
  float* p = static_cast<float*>(base) + at;
  if (FULL) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = f[i];
  }
}
template <bool FULL>
__device__ __forceinline__ uint2 load_codes(const void* base, long long at, int n) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + at;
  if (FULL) return __ldcs(reinterpret_cast<const uint2*>(p));
  uint32_t r[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) r[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint2(r[0], r[1]);
}
__device__ __forceinline__ void decode(const uint2& q, float scale, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? q.x : q.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w >> (16 * (i & 1))), __NV_E4M3);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = x.x * scale;
    f[2 * i + 1] = x.y * scale;
  }
}
// The larger magnitude, NaN if one of the two is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Square root, within 1 ulp, subnormals included.
__device__ __forceinline__ float sqrt_fast(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The codes of 8 values of a block whose scale this also writes. ROOT: the
// values are square roots, none negative, and what is not zero gets at least
// the smallest code.
template <bool FULL, bool ROOT>
__device__ __forceinline__ void store_codes(void* base, float* scale, long long at, int n,
                                            const float* f) {
  float top = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = max_nan(top, fabsf(f[i]));
  // magnitudes compare as integers, and a NaN is larger than everything
  const float big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu));
  const bool tiny = big < 7.888609052210118e-31f;  // 2^-100: 448 / big stays finite
  const float inv = tiny ? 0.f : __fdividef(448.f, big);
  uint32_t r[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = f[2 * i] * inv, b = f[2 * i + 1] * inv;
    if (ROOT) {  // above 2^-10, half the smallest code, rounding goes up
      if (a > 0.f) a = fmaxf(a, 0.001f);
      if (b > 0.f) b = fmaxf(b, 0.001f);
    }
    r[i / 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3))
                << (16 * (i & 1));
  }
  uint8_t* p = static_cast<uint8_t*>(base) + at;
  if (FULL) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(r[0], r[1]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(r[i / 4] >> (8 * (i & 3)));
  }
  // an infinite or NaN maximum makes the scale, and with it the block, NaN
  if ((threadIdx.x & 31) == 0)
    *scale = tiny ? 0.f : (big <= 3.402823466e+38f ? big / 448.f : __int_as_float(0x7fc00000));
}

struct AdamStep {
  float lr, step, inv2, gs;  // rate, rate / (1 - beta1^t), 1 / sqrt(1 - beta2^t), gradient scale
};

// One block of one tensor; PF32, MASTER, GF32, Q8: the tensor's types.
template <bool PF32, bool MASTER, bool GF32, bool Q8, bool FULL>
__device__ __forceinline__ void adam_block(const AdamParams& P, const AdamTensor& t, const AdamStep& h,
                                           long long blk, long long at, int n) {
  float p[8], g[8], m[8], v[8], root[8];
  uint2 qm, qv;
  float sm, sv;
  if (Q8) {
    qm = load_codes<FULL>(t.m, at, n), qv = load_codes<FULL>(t.v, at, n);
    sm = t.m_scale[blk], sv = t.v_scale[blk];
  } else {
    load_f32<FULL>(t.m, at, n, m);
    load_f32<FULL>(t.v, at, n, v);
  }
  if (GF32) load_f32<FULL>(t.g, at, n, g);
  else load_bf16<FULL>(t.g, at, n, g);
  if (MASTER) load_f32<FULL>(t.master, at, n, p);
  else if (PF32) load_f32<FULL>(t.p, at, n, p);
  else load_bf16<FULL>(t.p, at, n, p);
  if (Q8) {
    decode(qm, sm, m);
    decode(qv, sv, v);
  }
  const float keep = 1.f - h.lr * t.wd;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = g[i] * h.gs;
    m[i] = P.b1 * m[i] + P.b1c * gi;
    const float vi = Q8 ? v[i] * v[i] : v[i];
    v[i] = P.b2 * vi + P.b2c * (gi * gi);
    root[i] = sqrt_fast(v[i]);
    p[i] = p[i] * keep - h.step * __fdividef(m[i], root[i] * h.inv2 + P.eps);
    if (!FULL && i >= n) m[i] = root[i] = 0.f;  // what does not exist has no part in a maximum
  }
  if (MASTER) store_f32<FULL>(t.master, at, n, p);
  if (PF32) store_f32<FULL>(t.p, at, n, p);
  else store_bf16<FULL>(t.p, at, n, p);
  if (Q8) {
    store_codes<FULL, false>(t.m, t.m_scale + blk, at, n, m);
    store_codes<FULL, true>(t.v, t.v_scale + blk, at, n, root);
  } else {
    store_f32<FULL>(t.m, at, n, m);
    store_f32<FULL>(t.v, at, n, v);
  }
}

template <bool PF32, bool MASTER, bool GF32, bool Q8>
__device__ __forceinline__ void adam_any(const AdamParams& P, const AdamTensor& t, const AdamStep& h,
                                         long long blk, int lane) {
  const long long at = blk * kBlock + lane * 8;
  if ((blk + 1) * kBlock <= t.n)
    adam_block<PF32, MASTER, GF32, Q8, true>(P, t, h, blk, at, 8);
  else
    adam_block<PF32, MASTER, GF32, Q8, false>(P, t, h, blk, at,
                                              static_cast<int>(max(0LL, min(8LL, t.n - at))));
}

__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamParams P) {
  float lr = P.lr, c1 = P.c1, rc2 = P.rc2, gs = P.gs;
  if (P.dyn != nullptr) lr = P.dyn[0], c1 = P.dyn[1], rc2 = P.dyn[2], gs = P.dyn[3];
  const AdamStep h = {lr, lr / c1, 1.f / rc2, gs};
  const int lane = threadIdx.x & 31;
  const long long total = P.first[P.count];
  const long long warps = static_cast<long long>(gridDim.x) * (kAdamThreads / 32);
  int k = 0;
  for (long long b = static_cast<long long>(blockIdx.x) * (kAdamThreads / 32) + threadIdx.x / 32;
       b < total; b += warps) {
    if (b >= P.first[k + 1]) {  // the tensor that holds block b
      int hi = P.count;
      while (hi - k > 1) {
        const int mid = (k + hi) / 2;
        if (P.first[mid] <= b) k = mid; else hi = mid;
      }
    }
    const AdamTensor& t = P.t[k];
    const long long blk = b - P.first[k];
    switch (t.types) {
#define ADAM_CASE(p, m, g, q) \
  case (p) | (m) << 1 | (g) << 2 | (q) << 3: adam_any<p, m, g, q>(P, t, h, blk, lane); break
      ADAM_CASE(0, 0, 0, 0);
      ADAM_CASE(0, 0, 0, 1);
      ADAM_CASE(0, 0, 1, 0);
      ADAM_CASE(0, 0, 1, 1);
      ADAM_CASE(0, 1, 0, 0);
      ADAM_CASE(0, 1, 0, 1);
      ADAM_CASE(0, 1, 1, 0);
      ADAM_CASE(0, 1, 1, 1);
      ADAM_CASE(1, 0, 0, 0);
      ADAM_CASE(1, 0, 0, 1);
      ADAM_CASE(1, 0, 1, 0);
      ADAM_CASE(1, 0, 1, 1);
#undef ADAM_CASE
    }
  }
}

}  // namespace

cudaError_t launch_adamw(const moe_adamw_cfg& c, const moe_adamw_tensor* t, int n, cudaStream_t s) {
  AdamParams P;
  P.dyn = c.dyn;
  P.lr = static_cast<float>(c.lr);
  P.c1 = static_cast<float>(1.0 - pow(c.beta1, static_cast<double>(c.step)));
  P.rc2 = static_cast<float>(sqrt(1.0 - pow(c.beta2, static_cast<double>(c.step))));
  P.gs = static_cast<float>(c.grad_scale);
  P.b1 = static_cast<float>(c.beta1);
  P.b1c = static_cast<float>(1.0 - c.beta1);
  P.b2 = static_cast<float>(c.beta2);
  P.b2c = static_cast<float>(1.0 - c.beta2);
  P.eps = static_cast<float>(c.eps);
  for (int i = 0; i < n;) {
    P.count = 0;
    P.first[0] = 0;
    for (; i < n && P.count < kMaxTensors; ++i) {
      if (t[i].n == 0) continue;
      AdamTensor& o = P.t[P.count];
      o.p = t[i].p, o.master = t[i].master, o.g = t[i].g, o.m = t[i].m, o.v = t[i].v;
      o.m_scale = t[i].m_scale, o.v_scale = t[i].v_scale, o.n = t[i].n;
      o.wd = static_cast<float>(c.weight_decay * t[i].wd_scale);
      o.types = (t[i].p_type == MOE_T_F32 ? 1 : 0) | (t[i].master != nullptr ? 2 : 0) |
                (t[i].g_type == MOE_T_F32 ? 4 : 0) | (t[i].state_type == MOE_STATE_8BIT ? 8 : 0);
      P.first[P.count + 1] = P.first[P.count] + (o.n + kBlock - 1) / kBlock;
      ++P.count;
    }
    if (P.count == 0) break;
    const long long ctas = (P.first[P.count] + kAdamThreads / 32 - 1) / (kAdamThreads / 32);
    const int grid = static_cast<int>(ctas < num_sms() * 8LL ? ctas : num_sms() * 8LL);
    adamw_kernel<<<grid, kAdamThreads, 0, s>>>(P);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sgl
