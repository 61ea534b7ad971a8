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
  int types; // bit 0: p fp32, bit 1: g fp32, bit 2: 8-bit states
};

struct AdamParams {
  int count;
  float lr, c1, rc2, gs;  // rate, 1 - beta1^t, sqrt(1 - beta2^t), gradient scale
  float b1, b1c, b2, b2c, eps;
  const float* dyn;
  long long first[kMaxTensors + 1];  // prefix sums of the tensors' blocks
  AdamTensor t[kMaxTensors];
};

// n: elements of this lane's piece that exist (8 or fewer)
__device__ __forceinline__ void load_bf16(const void* base, long long at, int n, float* f) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  if (n == 8) {
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
__device__ __forceinline__ void load_f32(const void* base, long long at, int n, float* f) {
  const float* p = static_cast<const float*>(base) + at;
  if (n == 8) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.f;
  }
}
__device__ __forceinline__ void store_bf16(void* base, long long at, int n, const float* f) {
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if (n == 8) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(r[0], r[1], r[2], r[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(r[i / 2] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store_f32(void* base, long long at, int n, const float* f) {
  float* p = static_cast<float*>(base) + at;
  if (n == 8) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = f[i];
  }
}
// 8 e4m3 codes times the block's scale
__device__ __forceinline__ void load_codes(const void* base, long long at, int n, float scale, float* f) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + at;
  uint32_t r[2] = {0, 0};
  if (n == 8) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
    r[0] = v.x, r[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) r[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(r[i / 2] >> (16 * (i & 1))), __NV_E4M3);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = x.x * scale;
    f[2 * i + 1] = x.y * scale;
  }
}
// The codes of 8 values of a block whose scale this also writes. FLOOR: what
// is not zero gets at least the smallest code.
template <bool FLOOR>
__device__ __forceinline__ void store_codes(void* base, float* scale, long long blk, long long at,
                                            int n, const float* f) {
  // magnitudes compare as integers, and a NaN is larger than everything
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  const float big = __uint_as_float(top);
  const bool tiny = big < 7.888609052210118e-31f;  // 2^-100: 448 / big stays finite
  const float inv = tiny ? 0.f : 448.f / big;
  uint32_t r[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = f[2 * i] * inv, b = f[2 * i + 1] * inv;
    uint32_t q = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    if (FLOOR) {
      if (a > 0.f && (q & 0xffu) == 0) q |= 1u;
      if (b > 0.f && (q & 0xff00u) == 0) q |= 0x100u;
    }
    r[i / 2] |= q << (16 * (i & 1));
  }
  uint8_t* p = static_cast<uint8_t*>(base) + at;
  if (n == 8) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(r[0], r[1]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(r[i / 4] >> (8 * (i & 3)));
  }
  // an infinite or NaN maximum makes the scale, and with it the block, NaN
  if ((threadIdx.x & 31) == 0)
    scale[blk] = tiny ? 0.f : (top >= 0x7f800000u ? __int_as_float(0x7fc00000) : big / 448.f);
}

__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamParams P) {
  float lr = P.lr, c1 = P.c1, rc2 = P.rc2, gs = P.gs;
  if (P.dyn != nullptr) lr = P.dyn[0], c1 = P.dyn[1], rc2 = P.dyn[2], gs = P.dyn[3];
  const float step = lr / c1, inv2 = 1.f / rc2;
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
    const long long blk = b - P.first[k], at = blk * kBlock + lane * 8;
    const int n = static_cast<int>(max(0LL, min(8LL, t.n - at)));
    float p[8], g[8], m[8], v[8];
    if (t.master != nullptr) load_f32(t.master, at, n, p);
    else if (t.types & 1) load_f32(t.p, at, n, p);
    else load_bf16(t.p, at, n, p);
    if (t.types & 2) load_f32(t.g, at, n, g);
    else load_bf16(t.g, at, n, g);
    const bool q8 = (t.types & 4) != 0;
    if (q8) {
      load_codes(t.m, at, n, t.m_scale[blk], m);
      load_codes(t.v, at, n, t.v_scale[blk], v);
    } else {
      load_f32(t.m, at, n, m);
      load_f32(t.v, at, n, v);
    }
    const float keep = 1.f - lr * t.wd;
    float root[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gi = g[i] * gs;
      m[i] = P.b1 * m[i] + P.b1c * gi;
      const float vi = q8 ? v[i] * v[i] : v[i];
      v[i] = P.b2 * vi + P.b2c * (gi * gi);
      root[i] = sqrtf(v[i]);
      p[i] = p[i] * keep - step * __fdividef(m[i], root[i] * inv2 + P.eps);
    }
    if (t.master != nullptr) store_f32(t.master, at, n, p);
    if (t.types & 1) store_f32(t.p, at, n, p);
    else store_bf16(t.p, at, n, p);
    if (q8) {
      if (n < 8) {  // lanes past the end do not count for the maximum
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= n) m[i] = 0.f, root[i] = 0.f;
      }
      store_codes<false>(t.m, t.m_scale, blk, at, n, m);
      store_codes<true>(t.v, t.v_scale, blk, at, n, root);
    } else {
      store_f32(t.m, at, n, m);
      store_f32(t.v, at, n, v);
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
      o.types = (t[i].p_type == MOE_T_F32 ? 1 : 0) | (t[i].g_type == MOE_T_F32 ? 2 : 0) |
                (t[i].state_type == MOE_STATE_8BIT ? 4 : 0);
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
