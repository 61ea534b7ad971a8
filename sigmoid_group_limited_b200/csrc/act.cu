// act.cu - SwiGLU with its limit and routing weight, forward and backward
// (moe_swiglu, moe_swiglu_backward).
//
//   a = clamp(g), b = clamp(u), s = 1 / (1 + e^-a)
//   h  = w a s b
//   dg = w dh b (s + a s (1 - s)) where |g| <= limit, else 0
//   du = w dh a s                 where |u| <= limit, else 0
//   dw = sum_i dh a s b
//
// Both are bound by memory: 6 bytes per element forward (g, u in, h out), 10
// backward; 32768 x 768 take 28.5 us (5.3 TB/s) and 48.3 us (5.2 TB/s), launch
// included. Fewer or more pieces under way per lane, two to six blocks an SM
// and the next row's weight loaded ahead change that by less than 5 %. A group of G
// lanes owns a row (so dw is one shuffle reduction, in a fixed order) and moves 8
// features (16 bytes) per lane and tensor; rows wider than 2048 take a block each
// (8192 x 4096, in a graph: 34.7 us forward, 60.1 backward, 5.8 and 5.6 TB/s).
// Everything between the loads and the one rounding of each output is fp32;
// the exponential is the hardware one (see sigmoid_fast for its error, which is
// largest, 5e-6, where it counts least; bf16's half step is 2^-8).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace sgl {
namespace {

constexpr int kActThreads = 256;

struct ActParams {
  int R, chunks;  // rows, 8-feature pieces per row
  long long ld_g, ld_h, ld_dg;
  float limit;  // inf: off
  const uint16_t *dh, *g, *u;
  const float* w;
  const int32_t* perm;
  int n_w;
  const int32_t* rows;
  uint16_t *h, *dg, *du;
  float* dw;
};

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r[i] << 16);
    f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ uint4 load8(const uint16_t* p, long long at) {
  return __ldcs(reinterpret_cast<const uint4*>(p + at));
}
__device__ __forceinline__ void store8(uint16_t* p, long long at, const uint4& v) {
  *reinterpret_cast<uint4*>(p + at) = v;
}
// The limit, keeping a NaN (fminf / fmaxf would drop it).
__device__ __forceinline__ float clamp_nan(float v, float L) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(L));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(-L));
  return r;
}
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// s = 1 / (1 + e^-a). The exponential's relative error is about (|a| + 2) 2^-24,
// from the rounding of its argument, and counts by 1 - s. Below kFarGate (DEEP)
// s is at the end of fp32's normal numbers or below, where 1 + e^-a overflows
// and the reciprocal is cut to zero, but s a is still a number that bf16 holds:
// there s = e^a, formed 2^24 times too large (spacing 2^-149, zero from -104 on).
constexpr float kFarGate = -87.f, kLog2e = 1.44269504f;
template <bool DEEP>
__device__ __forceinline__ float sigmoid_fast(float a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_fast(-kLog2e * a)));
  if (DEEP && a < kFarGate) r = exp2_fast(fmaf(kLog2e, a, 24.f)) * 5.9604644775390625e-8f;
  return r;
}
// The least of 8 bf16 values (of those that are not NaN).
__device__ __forceinline__ float least8(const uint4& v) {
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&v);
  const float2 m = __bfloat1622float2(__hmin2(__hmin2(b[0], b[1]), __hmin2(b[2], b[3])));
  return fminf(m.x, m.y);
}

// Routing weight of row r and where its gradient goes (-1: nowhere).
__device__ __forceinline__ float row_weight(const ActParams& p, int r, long long* slot) {
  *slot = -1;
  if (p.w == nullptr) return 1.f;
  long long j = r;
  if (p.perm != nullptr) {
    j = p.perm[r];
    if (j < 0 || j >= p.n_w) return __int_as_float(0x7fc00000);
  }
  *slot = j;
  return p.w[j];
}

// A group of G lanes owns a row, and each lane has U pieces of it under way:
// with four blocks to an SM about 100 KB of loads.
template <int G, bool BWD>
__global__ void __launch_bounds__(kActThreads, 4) act_kernel(const ActParams p) {
  constexpr int U = BWD ? 2 : 4;
  pdl_wait();
  const int live = p.rows ? max(0, min(*p.rows, p.R)) : p.R;
  const int lane = threadIdx.x % G;
  const int per = kActThreads / G;
  for (int r = blockIdx.x * per + threadIdx.x / G; r < live; r += gridDim.x * per) {
    long long slot;
    const float w = row_weight(p, r, &slot);
    float sum = 0.f;
    for (int c0 = lane; c0 < p.chunks; c0 += G * U) {
      uint4 qg[U], qu[U], qd[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int c = c0 + k * G;
        if (c < p.chunks) {
          qg[k] = load8(p.g, r * p.ld_g + 8 * c);
          qu[k] = load8(p.u, r * p.ld_g + 8 * c);
          if (BWD) qd[k] = load8(p.dh, r * p.ld_h + 8 * c);
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int c = c0 + k * G;
        if (c >= p.chunks) break;
        float g[8], u[8], dh[8], o[8], o2[8];
        unpack8(qg[k], g);
        unpack8(qu[k], u);
        if (BWD) unpack8(qd[k], dh);
        auto compute = [&](auto deep) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = clamp_nan(g[i], p.limit), b = clamp_nan(u[i], p.limit);
            const float s = sigmoid_fast<decltype(deep)::value>(a);
            const float silu = a * s;
            if (!BWD) {
              o[i] = w * silu * b;
            } else {
              sum += dh[i] * (silu * b);
              const float wd = w * dh[i];
              o[i] = fabsf(g[i]) > p.limit ? 0.f : wd * b * (s + silu * (1.f - s));
              o2[i] = fabsf(u[i]) > p.limit ? 0.f : wd * silu;
            }
          }
        };
        if (least8(qg[k]) < kFarGate && p.limit > -kFarGate) compute(std::true_type());  // rare
        else compute(std::false_type());
        if (!BWD) {
          store8(p.h, r * p.ld_h + 8 * c, pack8(o));
        } else {
          store8(p.dg, r * p.ld_dg + 8 * c, pack8(o));
          store8(p.du, r * p.ld_dg + 8 * c, pack8(o2));
        }
      }
    }
    if (BWD && p.dw != nullptr) {
      constexpr int W = G < 32 ? G : 32;
      // the lanes of this row (other rows of the warp may have ended)
      const uint32_t mask = W == 32 ? 0xffffffffu : ((1u << W) - 1u) << (threadIdx.x % 32 / W * W);
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o, W);
      if (G > 32) {  // the whole block is in this row
        __shared__ float part[kActThreads / 32];
        __syncthreads();
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
        __syncthreads();
        sum = 0.f;
        for (int i = 0; i < kActThreads / 32; ++i) sum += part[i];
      }
      if (lane == 0 && slot >= 0) p.dw[slot] = sum;
    }
  }
}

template <int G, bool BWD>
cudaError_t launch_rows(const ActParams& p, cudaStream_t s) {
  const int grid = min(cdiv(p.R, kActThreads / G), num_sms() * 8);
  return launch_pdl(act_kernel<G, BWD>, dim3(grid), dim3(kActThreads), 0, s, p);
}

template <bool BWD>
cudaError_t launch_act(const ActParams& p, cudaStream_t s) {
  if (p.chunks <= 32) return launch_rows<8, BWD>(p, s);
  if (p.chunks <= 256) return launch_rows<32, BWD>(p, s);
  return launch_rows<kActThreads, BWD>(p, s);
}

ActParams common(const moe_swiglu_desc& d, const void* g, const void* u, const float* w,
                 const int32_t* perm, int n_w, const int32_t* rows) {
  ActParams p = {};
  p.R = d.R;
  p.chunks = d.I / 8;
  p.ld_g = d.ld_g;
  p.ld_h = d.ld_h;
  p.ld_dg = d.ld_dg;
  p.limit = d.limit > 0.f ? d.limit : INFINITY;
  p.g = static_cast<const uint16_t*>(g);
  p.u = static_cast<const uint16_t*>(u);
  p.w = w;
  p.perm = perm;
  p.n_w = n_w;
  p.rows = rows;
  return p;
}

}  // namespace

cudaError_t launch_swiglu(const moe_swiglu_desc& d, const void* g, const void* u, const float* w,
                          const int32_t* perm, int n_w, const int32_t* rows, void* h,
                          cudaStream_t s) {
  ActParams p = common(d, g, u, w, perm, n_w, rows);
  p.h = static_cast<uint16_t*>(h);
  return launch_act<false>(p, s);
}

cudaError_t launch_swiglu_backward(const moe_swiglu_desc& d, const void* dh, const void* g,
                                   const void* u, const float* w, const int32_t* perm, int n_w,
                                   const int32_t* rows, void* dg, void* du, float* dw,
                                   cudaStream_t s) {
  ActParams p = common(d, g, u, w, perm, n_w, rows);
  p.dh = static_cast<const uint16_t*>(dh);
  p.dg = static_cast<uint16_t*>(dg);
  p.du = static_cast<uint16_t*>(du);
  p.dw = dw;
  return launch_act<true>(p, s);
}

}  // namespace sgl
