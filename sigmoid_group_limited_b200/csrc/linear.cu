// linear.cu - products grouped by expert with ragged row counts
// (moe_grouped_linear and its two gradients).
//
//   forward  y[r,n]    = sum_k x[r,k]  W[e,n,k]      rows r of expert e
//   dgrad    dx[r,k]   = sum_n dy[r,n] W[e,n,k]
//   wgrad    dW[e,n,k] = sum_r dy[r,n] x[r,k]
//
// The simple form: 64 x 64 output tiles, fp32 fused multiply-adds.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace sgl {
namespace {

constexpr int kTile = 64, kDeep = 16, kThreads = 256;

struct LinParams {
  int E, R, N, K;
  long long ld_x, ld_y;
  int out_f32, accumulate;
  const uint16_t *a, *b;
  const int32_t* offsets;
  void* out;
  int32_t* err;
};

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// Rows [lo, hi) of expert e, held inside [0, R] whatever the offsets say.
__device__ __forceinline__ int2 expert_range(const LinParams& p, int e) {
  const int a = p.offsets[e], b = p.offsets[e + 1];
  if (a < 0 || b < a || b > p.R) atomicExch(p.err, MOE_DEVERR_OFFSETS);
  const int lo = min(max(a, 0), p.R);
  return make_int2(lo, min(max(b, lo), p.R));
}

template <int DIR>
__global__ void __launch_bounds__(kThreads) linear_simple(const LinParams p) {
  __shared__ float sa[kDeep][kTile + 1], sb[kDeep][kTile + 1];
  const int cols = DIR == kFwd ? p.N : p.K;
  const int c0 = blockIdx.y * kTile;
  int e = blockIdx.z, lo = 0, hi = 0, m0 = 0, m_end = 0;
  if (DIR == kWgrad) {
    const int2 r = expert_range(p, e);
    lo = r.x, hi = r.y;
    m0 = blockIdx.x * kTile, m_end = p.N;
  } else {  // blockIdx.x: a 64-row tile, counted over the experts
    int left = blockIdx.x;
    for (e = 0; e < p.E; ++e) {
      const int2 r = expert_range(p, e);
      const int tiles = (r.y - r.x + kTile - 1) / kTile;
      if (left < tiles) {
        m0 = r.x + left * kTile, m_end = r.y;
        break;
      }
      left -= tiles;
    }
    if (e == p.E) return;
    hi = DIR == kFwd ? p.K : p.N;
  }
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = lo; k0 < hi; k0 += kDeep) {
    for (int i = threadIdx.x; i < kTile * kDeep; i += kThreads) {
      const int t = i % kTile, d = k0 + i / kTile;
      float av = 0.f, bv = 0.f;
      if (d < hi) {
        if (m0 + t < m_end)
          av = DIR == kWgrad ? bf(p.a[d * p.ld_y + m0 + t])
                             : bf(p.a[(m0 + t) * (DIR == kFwd ? p.ld_x : p.ld_y) + d]);
        if (c0 + t < cols)
          bv = DIR == kWgrad ? bf(p.b[d * p.ld_x + c0 + t])
               : DIR == kFwd ? bf(p.b[(static_cast<long long>(e) * p.N + c0 + t) * p.K + d])
                             : bf(p.b[(static_cast<long long>(e) * p.N + d) * p.K + c0 + t]);
      }
      sa[i / kTile][t] = av;
      sb[i / kTile][t] = bv;
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[d][ty * 4 + i] * sb[d][tx * 4 + j];
    __syncthreads();
  }
  if (DIR == kWgrad && lo == hi && p.accumulate) return;
  const long long ld = DIR == kFwd ? p.ld_y : DIR == kDgrad ? p.ld_x : p.K;
  const long long row0 = DIR == kWgrad ? static_cast<long long>(e) * p.N : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, c = c0 + tx * 4 + j;
      if (m >= m_end || c >= cols) continue;
      const long long at = (row0 + m) * ld + c;
      if (p.out_f32) {
        float* o = static_cast<float*>(p.out) + at;
        *o = p.accumulate ? *o + acc[i][j] : acc[i][j];
      } else {
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(acc[i][j]);
      }
    }
}

}  // namespace

cudaError_t launch_grouped_linear(const moe_linear_desc& d, LinearDir dir, const void* a,
                                  const void* b, const int32_t* offsets, void* out, int32_t* err,
                                  cudaStream_t s) {
  LinParams p = {d.E, d.R, d.N, d.K, d.ld_x, d.ld_y, d.out_type == MOE_T_F32, d.accumulate != 0,
                 static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), offsets, out, err};
  const int cols = dir == kFwd ? d.N : d.K;
  const int row_tiles = cdiv(d.R, kTile) + min(d.E, d.R);
  const dim3 rows(row_tiles, cdiv(cols, kTile), 1), weights(cdiv(d.N, kTile), cdiv(cols, kTile), d.E);
  if (dir == kFwd) linear_simple<kFwd><<<rows, kThreads, 0, s>>>(p);
  else if (dir == kDgrad) linear_simple<kDgrad><<<rows, kThreads, 0, s>>>(p);
  else linear_simple<kWgrad><<<weights, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace sgl
