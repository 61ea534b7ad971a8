// adamw.cu - one AdamW step over many tensors (moe_adamw_step), states in
// fp32 or in 8 bits.
//
// Bound by HBM: 28 bytes per element with fp32 states, a bf16 parameter, its
// master and a bf16 gradient; 10.06 with 8-bit states and no master. One
// launch takes as many tensors as its parameter block holds; the work is the
// list of all tensors' 256-element blocks, a warp per block (8 elements, 16
// bytes of bf16, per lane), so a block's maximum for the 8-bit scales is one
// warp reduction and nothing is read twice. No atomics: an element is owned
// by one lane. The arithmetic of 8-bit states fills most of the issue slots
// (44 instructions an element), so it is kept short: the scales go into the
// moments' coefficients, and roots and reciprocals are the hardware's.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace sgl {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kBlock = MOE_STATE_BLOCK;  // 32 lanes x 8 elements
// Most blocks a warp takes at a time. Starting on a tensor (its pointers, the
// first loads with nothing to compute meanwhile) costs about as much as a few
// blocks: 8-bit states over 377 M elements took 989, 893, 708 and 732 us with
// 1, 8, 32 and 64. Fewer where warps would be left without work.
constexpr int kSpan = 32;
// Tensors per launch: a parameter block of 3 KB, or of 26 KB for longer lists
// (240 small tensors: 11.6 us in one launch, 22 us in launches of 40).
constexpr int kFewTensors = 32, kManyTensors = 320;
constexpr int kAdamCtas = 3;  // per SM; at 4 the wider types spill (690 for 597 us)

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
  int types; // bit 0: p fp32, bit 1: master, bit 2: g fp32
};

template <int CAP>
struct AdamParams {
  int count;
  float lr, c1, rc2, gs;  // rate, 1 - beta1^t, sqrt(1 - beta2^t), gradient scale
  float b1, b1c, b2, b2c, eps;
  const float* dyn;
  int span;                          // blocks of a unit of work
  long long first[CAP + 1];          // prefix sums of the tensors' units
  AdamTensor t[CAP];
};
static_assert(sizeof(AdamParams<kManyTensors>) <= 32764, "kernel parameters");

// A lane's piece of 8 elements of B bytes as 2 B words. Of a tensor's last
// block only n of the 8 exist; the others read as zero and are not written.
template <int B>
struct Piece {
  uint32_t w[2 * B];
};
template <int B>
__device__ __forceinline__ Piece<B> load_piece(const void* base, long long at, int n) {
  Piece<B> r;
  const uint8_t* p = static_cast<const uint8_t*>(base) + at * B;
  if (n == 8) {
    if (B == 1) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
      r.w[0] = v.x, r.w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < B / 2; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * B; ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if (B == 1) r.w[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
        else if (B == 2) r.w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i & 1));
        else r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
  }
  return r;
}
template <int B>
__device__ __forceinline__ void store_piece(void* base, long long at, int n, const Piece<B>& r) {
  uint8_t* p = static_cast<uint8_t*>(base) + at * B;
  if (n == 8) {
    if (B == 1) {
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(r.w[0], r.w[1]));
    } else {
#pragma unroll
      for (int i = 0; i < B / 2; ++i)
        __stcs(reinterpret_cast<uint4*>(p) + i,
               make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if (B == 1) p[i] = static_cast<uint8_t>(r.w[i / 4] >> (8 * (i & 3)));
        else if (B == 2) reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(r.w[i / 2] >> (16 * (i & 1)));
        else reinterpret_cast<uint32_t*>(p)[i] = r.w[i];
      }
  }
}
// fp32 values of a piece of fp32, bf16 or e4m3 elements, and back
__device__ __forceinline__ void unpack(const Piece<4>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void unpack(const Piece<2>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r.w[i] << 16);
    f[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Piece<1>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(r.w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
__device__ __forceinline__ void pack(const float* f, Piece<4>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(f[i]);
}
__device__ __forceinline__ void pack(const float* f, Piece<2>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
}
// The larger magnitude, NaN if one of the two is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Square root and reciprocal within about 1 ulp, subnormals taken as zero.
__device__ __forceinline__ float sqrt_fast(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The codes of 8 values of a block whose scale this also writes. ROOT: the
// values are square roots, none negative, and what is not zero gets at least
// the smallest code.
template <bool ROOT>
__device__ __forceinline__ void store_codes(void* base, float* scale, long long at, int n,
                                            const float* f) {
  float top = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = max_nan(top, fabsf(f[i]));
  // magnitudes compare as integers, and a NaN is larger than everything
  const float big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu));
  const bool tiny = big < 7.888609052210118e-31f;  // 2^-100: 448 / big stays finite
  const float inv = tiny ? 0.f : __fdividef(448.f, big);
  Piece<1> r = {{0, 0}};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.w[i / 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * inv, f[2 * i + 1] * inv),
                                                                 __NV_SATFINITE, __NV_E4M3))
                  << (16 * (i & 1));
  if (ROOT) {
    // a zero byte in one of the words (rare): is its value zero, too?
    const uint32_t z = ((r.w[0] - 0x01010101u) & ~r.w[0]) | ((r.w[1] - 0x01010101u) & ~r.w[1]);
    if ((z & 0x80808080u) != 0 && !tiny) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (f[i] > 0.f && (r.w[i / 4] >> (8 * (i & 3)) & 0xffu) == 0) r.w[i / 4] |= 1u << (8 * (i & 3));
    }
  }
  store_piece<1>(base, at, n, r);
  // an infinite or NaN maximum makes the scale, and with it the block, NaN
  if ((threadIdx.x & 31) == 0)
    *scale = tiny ? 0.f : (big <= 3.402823466e+38f ? big / 448.f : __int_as_float(0x7fc00000));
}

struct AdamStep {
  float lr, step, inv2;  // rate, rate / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float b1, b2, eps;
  float cg, cgg;         // (1 - beta1) and (1 - beta2) with the gradient scale and its square
};

// Blocks [blk, end) of one tensor; PF32, MASTER, GF32, Q8: its types. The next
// block's loads are under way while a block is computed.
template <bool PF32, bool MASTER, bool GF32, bool Q8>
__device__ __forceinline__ void adam_blocks(const AdamTensor& t, const AdamStep& h,
                                            long long blk, long long end, int lane) {
  struct Block {
    Piece<PF32 || MASTER ? 4 : 2> p;
    Piece<GF32 ? 4 : 2> g;
    Piece<Q8 ? 1 : 4> m, v;
    float sm, sv;
    int n;
  };
  const float keep = 1.f - h.lr * t.wd;
  auto load = [&](long long b) {
    Block k;
    const long long at = b * kBlock + lane * 8;
    k.n = static_cast<int>(max(0LL, min(8LL, t.n - at)));
    k.m = load_piece<Q8 ? 1 : 4>(t.m, at, k.n);
    k.v = load_piece<Q8 ? 1 : 4>(t.v, at, k.n);
    k.g = load_piece<GF32 ? 4 : 2>(t.g, at, k.n);
    k.p = load_piece<PF32 || MASTER ? 4 : 2>(MASTER ? t.master : t.p, at, k.n);
    if (Q8) k.sm = t.m_scale[b], k.sv = t.v_scale[b];
    return k;
  };
  Block next = load(blk);
#pragma unroll 1
  for (; blk < end; ++blk) {
    const Block k = next;
    if (Q8 && blk + 1 < end) next = load(blk + 1);
    const long long at = blk * kBlock + lane * 8;
    float p[8], g[8], m[8], v[8], root[8];
    unpack(k.p, p);
    unpack(k.g, g);
    unpack(k.m, m);
    unpack(k.v, v);
    // the moments' coefficients take the block's scales along
    const float cm = Q8 ? h.b1 * k.sm : h.b1, cv = Q8 ? h.b2 * (k.sv * k.sv) : h.b2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = cm * m[i] + h.cg * g[i];
      v[i] = cv * (Q8 ? v[i] * v[i] : v[i]) + h.cgg * (g[i] * g[i]);
      root[i] = sqrt_fast(v[i]);
      p[i] = p[i] * keep - h.step * (m[i] * rcp_fast(root[i] * h.inv2 + h.eps));
    }
    if (MASTER) {
      Piece<4> o;
      pack(p, o);
      store_piece<4>(t.master, at, k.n, o);
    }
    Piece<PF32 ? 4 : 2> o;
    pack(p, o);
    store_piece<PF32 ? 4 : 2>(t.p, at, k.n, o);
    if constexpr (Q8) {
      if (k.n < 8) {  // what does not exist has no part in a maximum
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= k.n) m[i] = root[i] = 0.f;
      }
      store_codes<false>(t.m, t.m_scale + blk, at, k.n, m);
      store_codes<true>(t.v, t.v_scale + blk, at, k.n, root);
    } else {
      Piece<4> w;
      pack(m, w);
      store_piece<4>(t.m, at, k.n, w);
      pack(v, w);
      store_piece<4>(t.v, at, k.n, w);
      if (blk + 1 < end) next = load(blk + 1);
    }
  }
}

template <bool Q8, int CAP>
__global__ void __launch_bounds__(kAdamThreads, kAdamCtas)
    adamw_kernel(const __grid_constant__ AdamParams<CAP> P) {
  pdl_wait();
  float lr = P.lr, c1 = P.c1, rc2 = P.rc2, gs = P.gs;
  if (P.dyn != nullptr) lr = P.dyn[0], c1 = P.dyn[1], rc2 = P.dyn[2], gs = P.dyn[3];
  const AdamStep h = {lr, lr / c1, 1.f / rc2, P.b1, P.b2, P.eps, P.b1c * gs, P.b2c * gs * gs};
  const int lane = threadIdx.x & 31;
  const long long total = P.first[P.count];
  const long long warps = static_cast<long long>(gridDim.x) * (kAdamThreads / 32);
  int k = 0;
  for (long long u = static_cast<long long>(blockIdx.x) * (kAdamThreads / 32) + threadIdx.x / 32;
       u < total; u += warps) {
    if (u >= P.first[k + 1]) {  // the tensor that holds unit u
      int hi = P.count;
      while (hi - k > 1) {
        const int mid = (k + hi) / 2;
        if (P.first[mid] <= u) k = mid; else hi = mid;
      }
    }
    const AdamTensor& t = P.t[k];
    const long long blk = (u - P.first[k]) * P.span;
    const long long end = min(blk + P.span, (t.n + kBlock - 1) / kBlock);
    switch (t.types) {
#define ADAM_CASE(p, m, g) \
  case (p) | (m) << 1 | (g) << 2: adam_blocks<p, m, g, Q8>(t, h, blk, end, lane); break
      ADAM_CASE(0, 0, 0);
      ADAM_CASE(0, 0, 1);
      ADAM_CASE(0, 1, 0);
      ADAM_CASE(0, 1, 1);
      ADAM_CASE(1, 0, 0);
      ADAM_CASE(1, 0, 1);
#undef ADAM_CASE
    }
  }
}

// The tensors with (Q8) or without 8-bit states, as many per launch as fit.
template <bool Q8, int CAP>
cudaError_t launch_states(AdamParams<CAP>& P, const moe_adamw_cfg& c, const moe_adamw_tensor* t, int n,
                          cudaStream_t s) {
  constexpr int warps = kAdamThreads / 32;
  for (int i = 0; i < n;) {
    P.count = 0;
    P.first[0] = 0;
    long long blocks = 0;
    for (; i < n && P.count < CAP; ++i) {
      if (t[i].n == 0 || (t[i].state_type == MOE_STATE_8BIT) != Q8) continue;
      AdamTensor& o = P.t[P.count++];
      o.p = t[i].p, o.master = t[i].master, o.g = t[i].g, o.m = t[i].m, o.v = t[i].v;
      o.m_scale = t[i].m_scale, o.v_scale = t[i].v_scale, o.n = t[i].n;
      o.wd = static_cast<float>(c.weight_decay * t[i].wd_scale);
      o.types = (t[i].p_type == MOE_T_F32 ? 1 : 0) | (t[i].master != nullptr ? 2 : 0) |
                (t[i].g_type == MOE_T_F32 ? 4 : 0);
      blocks += (o.n + kBlock - 1) / kBlock;
    }
    if (P.count == 0) break;
    const long long span = blocks / (2LL * num_sms() * kAdamCtas * warps);
    P.span = static_cast<int>(span < 1 ? 1 : span > kSpan ? kSpan : span);
    for (int k = 0; k < P.count; ++k)
      P.first[k + 1] = P.first[k] + (P.t[k].n + kBlock * P.span - 1) / (kBlock * P.span);
    // more CTAs than run at once: the late ones even out the early ones' ends
    const long long need = (P.first[P.count] + warps - 1) / warps, most = num_sms() * 8LL;
    const cudaError_t e = launch_pdl(adamw_kernel<Q8, CAP>, dim3(static_cast<unsigned>(need < most ? need : most)),
                                     dim3(kAdamThreads), 0, s, P);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int CAP>
cudaError_t launch_list(const moe_adamw_cfg& c, const moe_adamw_tensor* t, int n, cudaStream_t s) {
  AdamParams<CAP> P;
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
  const cudaError_t e = launch_states<false>(P, c, t, n, s);
  return e != cudaSuccess ? e : launch_states<true>(P, c, t, n, s);
}

}  // namespace

cudaError_t launch_adamw(const moe_adamw_cfg& c, const moe_adamw_tensor* t, int n, cudaStream_t s) {
  return n <= kFewTensors ? launch_list<kFewTensors>(c, t, n, s) : launch_list<kManyTensors>(c, t, n, s);
}

}  // namespace sgl
