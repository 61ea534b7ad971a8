// linear_few.cu - the forward grouped product for a few rows (decoding one or
// a few tokens): y[r,n] = sum_k x[r,k] W[e,n,k].
//
// With a handful of rows the product is the reading of the touched experts'
// weights, 2 N K bytes each, and on most experts a single row uses them. A
// tile of the tensor-core kernel (256 features) gives a token's 8 experts too
// few tiles for 148 SMs; here a block takes 8 to 32 features of one expert
// and up to 4 of its rows, so that those 8 experts make hundreds of equal
// units. A warp holds all of its features' weights (or 2560 elements of each
// at a time) in registers, straight from global memory and all under way at
// once, while the block brings the rows of x to shared memory. The sums are
// fp32, each lane over its pieces of K in order, then a butterfly over the
// lanes: the same bits every time.
//
// Bound by HBM from some 64 rows on. Rows of as many experts, 768 x 2560 weights,
// calls back to back in a graph, weights not in L2: 128 rows 83 us (6.1 TB/s), 64
// rows 44 us (5.7), a token's 8 rows (31 MB) 9.5 us against 4.9 at the copy rate. There
// the launch, the offsets' latency and 1.3 rounds of loads show (768 units on 592
// blocks, a second unit's loads starting after the first one's sums).
//
// A unit is named by its first row: the blocks fill a table [R] with the
// expert and the row count at every row that starts a unit, from one pass over
// the offsets, and need no prefix sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace sgl {
namespace {

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 4;      // rows of a unit

// Blocks per SM: more features need more registers for their sums.
__host__ __device__ constexpr int few_ctas(int features) { return features == 4 ? 3 : 4; }

struct FewParams {
  int E, R, N, K;
  long long ld_x, ld_y;
  int out_f32, accumulate;
  const uint16_t *x, *W;
  const int32_t* offsets;
  void* y;
  int32_t* err;
};

__device__ __forceinline__ void widen8(const uint4& q, float* f) {
  const uint32_t r[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r[i] << 16);
    f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}

// M rows from `row` on (expert e), features n .. n + F - 1 of this warp (on:
// they exist); P: pieces of 256 elements of a slab. Every warp of the block
// comes here together.
template <int F, int P, int M>
__device__ __forceinline__ void unit(const FewParams& p, uint16_t* xs, int e, int row, int n, bool on, int lane) {
  const uint16_t* w = p.W + (static_cast<long long>(e) * p.N + n) * p.K;
  float acc[M][F];
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[i][f] = 0.f;
  for (int s0 = 0; s0 < p.K; s0 += 256 * P) {
    uint4 q[P][F];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int k = s0 + 256 * j + lane * 8;
#pragma unroll
      for (int f = 0; f < F; ++f)
        q[j][f] = on && k < p.K ? __ldcs(reinterpret_cast<const uint4*>(w + static_cast<long long>(f) * p.K + k))
                                : make_uint4(0, 0, 0, 0);
    }
    // the rows' share of this slab, zeros past K
    for (int c = threadIdx.x; c < M * P * 32; c += kFewThreads) {
      const int i = c / (P * 32), k = s0 + (c - i * (P * 32)) * 8;
      reinterpret_cast<uint4*>(xs)[c] = k < p.K ? __ldg(reinterpret_cast<const uint4*>(p.x + (row + i) * p.ld_x + k))
                                                : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < P; ++j) {
      float wf[F][8];
#pragma unroll
      for (int f = 0; f < F; ++f) widen8(q[j][f], wf[f]);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        float x[8];
        widen8(reinterpret_cast<const uint4*>(xs)[(i * P + j) * 32 + lane], x);
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int t = 0; t < 8; ++t) acc[i][f] = fmaf(wf[f][t], x[t], acc[i][f]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int f = 0; f < F; ++f) {
      float s = acc[i][f];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (on && lane == i * F + f) {
        const long long at = (row + i) * p.ld_y + n + f;
        if (p.out_f32) {
          float* o = static_cast<float*>(p.y) + at;
          *o = p.accumulate ? *o + s : s;
        } else {
          static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16(s);
        }
      }
    }
}

// F features x P pieces that a warp holds: 10 to 12 loads per lane.
template <int F, int P>
__global__ void __launch_bounds__(kFewThreads, few_ctas(F)) grouped_linear_few(const FewParams p) {
  __shared__ int table[kFewMaxRows];  // at a unit's first row: expert * 8 + rows; else 0
  __shared__ __align__(16) uint16_t xs[kFewRows * P * 256];
  if (threadIdx.x < kFewMaxRows) table[threadIdx.x] = 0;
  pdl_wait();
  __syncthreads();
  bool bad = false;
  for (int e = threadIdx.x; e <= p.E; e += kFewThreads) {
    const int lo = p.offsets[e], hi = e < p.E ? p.offsets[e + 1] : p.R;
    if (lo < 0 || hi < lo || hi > p.R) {
      bad = true;
    } else if (e < p.E) {
      for (int r = lo; r < hi; r += kFewRows) table[r] = e * 8 + min(kFewRows, hi - r);
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicExch(p.err, MOE_DEVERR_OFFSETS);
    return;
  }
  const int lane = threadIdx.x & 31, wide = kFewWarps * F;
  const int cols = (p.N + wide - 1) / wide, units = p.R * cols;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int row = u / cols, n = (u - row * cols) * wide + static_cast<int>(threadIdx.x / 32) * F;
    const int t = table[row], e = t >> 3;
    switch (t & 7) {
      case 1: unit<F, P, 1>(p, xs, e, row, n, n < p.N, lane); break;
      case 2: unit<F, P, 2>(p, xs, e, row, n, n < p.N, lane); break;
      case 3: unit<F, P, 3>(p, xs, e, row, n, n < p.N, lane); break;
      case 4: unit<F, P, 4>(p, xs, e, row, n, n < p.N, lane); break;
    }
  }
}

template <int F, int P>
cudaError_t run(const FewParams& p, cudaStream_t s) {
  const int need = p.R * cdiv(p.N, kFewWarps * F), most = num_sms() * few_ctas(F);
  return launch_pdl(grouped_linear_few<F, P>, dim3(need < most ? need : most), dim3(kFewThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_linear_few(const moe_linear_desc& d, const void* x, const void* W,
                              const int32_t* offsets, void* y, int32_t* err, cudaStream_t s) {
  const FewParams p = {d.E, d.R, d.N, d.K, d.ld_x, d.ld_y, d.out_type == MOE_T_F32, d.accumulate != 0,
                       static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(W), offsets, y, err};
  // Short rows: more features per warp, so that as much is under way. A slab is 768,
  // 1280 or 2560 long, and a row just above a length pays for all of the next: 64 rows
  // of 768 features (timed as above) take 20 us with K = 1024, 23 with 1280, 35 with 1288, 36 with
  // 1536, 39 with 2048, 44 with 2560, 63 with 2568 and 67 with 3840.
  if (d.K <= 768) return run<4, 3>(p, s);
  if (d.K <= 1280) return run<2, 5>(p, s);
  return run<1, 10>(p, s);
}

}  // namespace sgl
