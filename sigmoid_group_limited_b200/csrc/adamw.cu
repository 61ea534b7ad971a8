// adamw.cu - one AdamW step over many tensors (moe_adamw_step), states in
// fp32 or in 8 bits.
//
// Bound by HBM: 28 bytes per element with fp32 states, a bf16 parameter, its
// master and a bf16 gradient; 10.06 with 8-bit states and no master. One
// launch takes as many tensors as its parameter block holds; the work is the
// list of all tensors' 256-element blocks, a warp per block (8 elements, 16
// bytes of bf16, per lane), so a block's maximum for the 8-bit scales is one
// warp reduction and nothing is read twice. No atomics: an element is owned
// by one lane. The arithmetic of 8-bit states fills most of the issue slots, so
// it is kept short: roots and reciprocals are the hardware's wherever they do
// not decide a code. 144 M elements with fp32 states: 668 us, 6.0 TB/s; 377 M
// with 8-bit states: 766 us sustained, 702 us in short runs, 5.0 to 5.4 TB/s at
// 58 instructions an element and 0.83 of the issue slots; with second moments that
// are all zero 938 us (see root_codes).
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
// 1, 8, 32 and 64 in the form they were chosen with. Fewer where warps would be
// left without work.
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
// block (not FULL) only n of the 8 exist; the others read as zero and are not
// written.
template <int B>
struct Piece {
  uint32_t w[2 * B];
};
template <int B, bool FULL>
__device__ __forceinline__ Piece<B> load_piece(const uint8_t* p, int n) {
  Piece<B> r;
  if (FULL) {
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
template <int B, bool FULL>
__device__ __forceinline__ void store_piece(uint8_t* p, int n, const Piece<B>& r) {
  if (FULL) {
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
// Square root and reciprocal within about 1 ulp; of a subnormal v the root is
// zero unless LOW (its root is a normal number), the reciprocal infinite.
template <bool LOW>
__device__ __forceinline__ float sqrt_fast(float v) {
  float r;
  if (LOW) asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  else asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The largest of 8 magnitudes of every lane (they compare as integers, and a
// NaN is larger than everything).
__device__ __forceinline__ float warp_max(const float* f) {
  float top = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = max_nan(top, fabsf(f[i]));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7fffffffu));
}
// The scales of a block's moments for their largest magnitudes, and the
// factors of their codes: lane 0 works on m, lane 1 on v.
__device__ __forceinline__ float2 write_scales(float* m_scale, float* v_scale, float top_m, float top_v) {
  const int lane = threadIdx.x & 31;
  const float top = lane == 0 ? top_m : top_v;
  const bool tiny = top < 7.888609052210118e-31f;  // 2^-100: the factor stays finite
  // an infinite or NaN maximum makes the scale, and with it the block, NaN
  if (lane < 2)
    *(lane == 0 ? m_scale : v_scale) =
        tiny ? 0.f : (top <= 3.402823466e+38f ? top * (1.f / 448.f) : __int_as_float(0x7fc00000));
  const float inv = tiny ? 0.f : __frcp_rn(top) * 448.f;
  return make_float2(__shfl_sync(0xffffffffu, inv, 0), __shfl_sync(0xffffffffu, inv, 1));
}
__device__ __forceinline__ Piece<1> to_codes(const float* y) {
  Piece<1> r = {{0, 0}};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.w[i / 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(y[2 * i], y[2 * i + 1]),
                                                                 __NV_SATFINITE, __NV_E4M3))
                  << (16 * (i & 1));
  return r;
}
// Codes of the square roots of 8 second moments. root: within an ulp or two,
// enough for a code unless the value lies at a border between two codes;
// there (low 19 mantissa bits near zero, 1 of 30000 values) the exact root
// decides, so that the codes are those of the definition. A zero counts as such a
// border, too, and costs its lane the exact roots. What is not zero gets at least
// the smallest code.
__device__ __forceinline__ Piece<1> root_codes(const float* v, const float* root, float inv) {
  float y[8];
  uint32_t near = 0x7ffffu;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = root[i] * inv;
    near = min(near, (__float_as_uint(y[i]) + 8u) & 0x7ffffu);
  }
  if (near < 16u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fsqrt_rn(v[i]) * inv;
  }
  Piece<1> r = to_codes(y);
  // a zero byte in one of the words (rare): is its value zero, too?
  const uint32_t z = ((r.w[0] - 0x01010101u) & ~r.w[0]) | ((r.w[1] - 0x01010101u) & ~r.w[1]);
  if ((z & 0x80808080u) != 0 && inv != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (y[i] > 0.f && (r.w[i / 4] >> (8 * (i & 3)) & 0xffu) == 0) r.w[i / 4] |= 1u << (8 * (i & 3));
  }
  return r;
}

struct AdamStep {
  float lr, step, inv2;  // rate, rate / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float b1, b2, eps;
  float b1c, b2c, gs;    // 1 - beta1, 1 - beta2, gradient scale
};

// `count` blocks of one tensor from blk on, all of them whole (FULL) or the one
// short block at its end; PF32, MASTER, GF32, Q8: its types; LOW: subnormal second
// moments count (see launch_list). With 8-bit states
// the next block's loads are under way while a block is computed.
template <bool PF32, bool MASTER, bool GF32, bool Q8, bool LOW, bool FULL>
__device__ __forceinline__ void adam_run(const AdamTensor& t, const AdamStep& h, long long blk, int count,
                                         int lane) {
  constexpr int BP = PF32 ? 4 : 2, BG = GF32 ? 4 : 2, BS = Q8 ? 1 : 4;
  struct Block {
    Piece<MASTER ? 4 : BP> p;
    Piece<BG> g;
    Piece<BS> m, v;
    float sm = 0.f, sv = 0.f;
  };
  const long long at = blk * kBlock + lane * 8;
  const int n = FULL ? 8 : static_cast<int>(max(0LL, min(8LL, t.n - at)));
  uint8_t* pp = static_cast<uint8_t*>(t.p) + at * BP;
  uint8_t* pw = MASTER ? reinterpret_cast<uint8_t*>(t.master + at) : pp;
  const uint8_t* pg = static_cast<const uint8_t*>(t.g) + at * BG;
  uint8_t *pm = static_cast<uint8_t*>(t.m) + at * BS, *pv = static_cast<uint8_t*>(t.v) + at * BS;
  float *ps = t.m_scale + blk, *pr = t.v_scale + blk;
  const float keep = 1.f - h.lr * t.wd;
  auto load = [&](int j) {  // block j from here on
    Block k;
    k.m = load_piece<BS, FULL>(pm + j * (kBlock * BS), n);
    k.v = load_piece<BS, FULL>(pv + j * (kBlock * BS), n);
    k.g = load_piece<BG, FULL>(pg + j * (kBlock * BG), n);
    k.p = load_piece<MASTER ? 4 : BP, FULL>(pw + j * (kBlock * (MASTER ? 4 : BP)), n);
    if (Q8) k.sm = ps[j], k.sv = pr[j];
    return k;
  };
  Block next;
  if (Q8) next = load(0);
#pragma unroll 1
  for (; count > 0; --count) {
    const Block k = Q8 ? next : load(0);
    if (Q8 && FULL && count > 1) next = load(1);
    float p[8], g[8], m[8], v[8], root[8];
    unpack(k.p, p);
    unpack(k.g, g);
    unpack(k.m, m);
    unpack(k.v, v);
    // The gradient is scaled before it is squared: under a scale that brings it
    // back into range neither g^2 nor the scale's square need fit fp32. (8-bit
    // states, 377 M elements: 766 us with this product, 759 without; a branch around
    // it for a scale of one: 764.)
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(h.gs, g[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (Q8) {
        // each operation rounded by itself: a code is a function of the
        // formula alone, and a run can be followed code by code
        const float mi = __fmul_rn(m[i], k.sm), ri = __fmul_rn(v[i], k.sv);
        m[i] = __fadd_rn(__fmul_rn(h.b1, mi), __fmul_rn(h.b1c, g[i]));
        v[i] = __fadd_rn(__fmul_rn(h.b2, __fmul_rn(ri, ri)), __fmul_rn(h.b2c, __fmul_rn(g[i], g[i])));
      } else {
        m[i] = h.b1 * m[i] + h.b1c * g[i];
        v[i] = h.b2 * v[i] + h.b2c * (g[i] * g[i]);
      }
      root[i] = sqrt_fast<LOW>(v[i]);
      p[i] = p[i] * keep - h.step * (m[i] * rcp_fast(root[i] * h.inv2 + h.eps));
    }
    if (MASTER) {
      Piece<4> o;
      pack(p, o);
      store_piece<4, FULL>(pw, n, o);
    }
    Piece<BP> o;
    pack(p, o);
    store_piece<BP, FULL>(pp, n, o);
    if constexpr (Q8) {
      if (!FULL) {  // what does not exist has no part in a maximum
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= n) m[i] = v[i] = root[i] = 0.f;
      }
      const float2 inv = write_scales(ps, pr, warp_max(m), __fsqrt_rn(warp_max(v)));
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = m[i] * inv.x;
      store_piece<1, FULL>(pm, n, to_codes(y));
      store_piece<1, FULL>(pv, n, root_codes(v, root, inv.y));
    } else {
      Piece<4> w;
      pack(m, w);
      store_piece<4, FULL>(pm, n, w);
      pack(v, w);
      store_piece<4, FULL>(pv, n, w);
    }
    pp += kBlock * BP, pg += kBlock * BG, pm += kBlock * BS, pv += kBlock * BS, ++ps, ++pr;
    pw += kBlock * (MASTER ? 4 : BP);
  }
}

// Blocks [blk, end) of one tensor.
template <bool PF32, bool MASTER, bool GF32, bool Q8, bool LOW>
__device__ __forceinline__ void adam_blocks(const AdamTensor& t, const AdamStep& h, long long blk,
                                            long long end, int lane) {
  const long long whole = min(end, t.n / kBlock);
  if (blk < whole) adam_run<PF32, MASTER, GF32, Q8, LOW, true>(t, h, blk, static_cast<int>(whole - blk), lane);
  if (whole < end) adam_run<PF32, MASTER, GF32, Q8, LOW, false>(t, h, whole, 1, lane);
}

template <bool Q8, bool LOW, int CAP>
__global__ void __launch_bounds__(kAdamThreads, kAdamCtas)
    adamw_kernel(const __grid_constant__ AdamParams<CAP> P) {
  pdl_wait();
  float lr = P.lr, c1 = P.c1, rc2 = P.rc2, gs = P.gs;
  if (P.dyn != nullptr) lr = P.dyn[0], c1 = P.dyn[1], rc2 = P.dyn[2], gs = P.dyn[3];
  const AdamStep h = {lr, lr / c1, 1.f / rc2, P.b1, P.b2, P.eps, P.b1c, P.b2c, gs};
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
  case (p) | (m) << 1 | (g) << 2: adam_blocks<p, m, g, Q8, LOW>(t, h, blk, end, lane); break
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
template <bool Q8, bool LOW, int CAP>
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
    const cudaError_t e = launch_pdl(adamw_kernel<Q8, LOW, CAP>, dim3(static_cast<unsigned>(need < most ? need : most)),
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
  // The root of a subnormal v, at most 2^-63, counts beside an eps below 2^24
  // times that (times the smallest sqrt(1 - beta2^step)). fp32 states, bound by memory, take
  // subnormals in their stride; 8-bit states, bound by issue, pay for them (377 M
  // elements 783 us for 751), so only a step with such an eps does.
  const bool low = c.eps * sqrt(1.0 - c.beta2) < 0x1p-39;
  const cudaError_t e = launch_states<false, true>(P, c, t, n, s);
  if (e != cudaSuccess) return e;
  return low ? launch_states<true, true>(P, c, t, n, s) : launch_states<true, false>(P, c, t, n, s);
}

}  // namespace

cudaError_t launch_adamw(const moe_adamw_cfg& c, const moe_adamw_tensor* t, int n, cudaStream_t s) {
  return n <= kFewTensors ? launch_list<kFewTensors>(c, t, n, s) : launch_list<kManyTensors>(c, t, n, s);
}

}  // namespace sgl
