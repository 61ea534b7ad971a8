// linear.cu - products grouped by expert with ragged row counts
// (moe_grouped_linear and its two gradients) on CTA pairs (tcgen05
// cta_group::2).
//
//   forward  y[r,n]    = sum_k x[r,k]  W[e,n,k]      rows r of expert e
//   dgrad    dx[r,k]   = sum_n dy[r,n] W[e,n,k]
//   wgrad    dW[e,n,k] = sum_r dy[r,n] x[r,k]
//
// One kernel, three sets of operands. A pair of CTAs (a cluster of two) owns
// an output tile D[256][up to 256] (128 columns where few tiles would leave
// pairs idle): M = 256 MMAs, each CTA with 128 rows of A
// and half of B's columns in its shared memory and 128 rows of D in its
// tensor memory. Forward and dgrad put the features (regular, hundreds) on M
// and an expert's rows (ragged) on N, so a short tile costs a narrower MMA,
// not a padded one; wgrad has features on both sides and the ragged rows as
// the contraction.
//
//   direction  M (A)                N (B)               contraction
//   forward    n: W, K-major        rows: x, K-major    k
//   dgrad      k: W, MN-major       rows: dy, K-major   n
//   wgrad      n: dy, MN-major      k: x, MN-major      rows
//
// MN-major operands are read in place: the TMA box is 64 features wide and 64
// contraction indices high, and the MMA transposes. The tensor maps end at
// the tensors' ends, so features past N or K read as zeros. Rows are another
// matter: behind an expert's rows come the next one's. On N they only fill
// columns that are never stored. In wgrad's contraction they must not count,
// whatever they hold: the last block runs only the 16-row steps that have
// rows, and a warp of each CTA zeroes the rest of the last step in shared
// memory (NaN times zero would be NaN) before the MMA may read the stage.
//
// Persistent: pair i takes tiles i, i + pairs, ...; every role finds its
// tiles from the row offsets by itself, so there is no queue, no counter and
// no state between calls, and the same call always adds in the same order.
// Two 256-column accumulators: a tile's epilogue runs under the next tile's
// MMAs.
//
// The tensor core's fp32 accumulation cuts low bits off at every step, always
// towards zero: per 16-deep step about 1.7e-8 of a sum of terms of both signs,
// 9e-8 where all have one sign (2.3 % at a depth of 4 M). So a contraction is
// made in passes, each in a fresh accumulator, added in fp32 (rounded to nearest).
//   fp32 results: passes of at most 768. The epilogue adds them to the output by
//   reductions in L2 (subnormals flushed; one per element and pass, by the same
//   thread in order, so the result is the same every time). A pass costs 6e-7 to
//   7.5e-7 of the result's norm whatever the depth, and the P adds at most P 2^-24:
//   7.4e-7 at a depth of 20011, 1.0e-6 at 1 M, 1.5e-6 at 4 M, 3.4e-6 at 2^25.
//   bf16 results: passes of at most 16384, about 1e-4 of the sum or 1/40 of the
//   final rounding; only wgrad is ever deeper. Their sum stays in tensor memory, in the
//   accumulator that the passes leave free, and is rounded once.
//
// What bounds it. Few rows per expert: the weights from HBM (512 experts, 768 x
// 2560, 32768 rows: 2.23 GB in 346 us, 6.4 TB/s). Hundreds of rows: an M = 256,
// N = 256 instruction takes 128 cycles and a 64-deep block four of them, while
// its 32 KB per SM need 512 cycles at the 64 bytes a clock that L2 delivers to
// an SM: the two meet, and the clock falls (to about 1.4 GHz) with the power
// that both draw. 64 uneven experts, 30011 rows: 113 us in short runs, 1.05
// PFLOP/s, 140 us sustained; the input gradient 120 and 149. A weight gradient
// writes as much as it reads: 160 us (fp32, 721 MB) and, for 512 experts of 64
// rows, 380 to 440 us (2.2 GB) depending on where its buffers lie.
//
// Tried and dropped: experts in order of their tiles' cost and equal tile
// widths (within 2 % either way); two accumulator chains (no difference);
// TMA boxes of 128 features (none); store hints, boxes of 128-byte rows and two
// boxes per warp (none, or the pipeline stage they cost).
//
// Warp roles per CTA (384 threads):
//   0      TMA producer (one lane)
//   1      TMEM allocation; MMA issuer (one lane) in the leader
//   2      wgrad: zeroes the rows behind an expert's last
//   3      idle
//   4..11  epilogue, two warps per TMEM lane quarter, alternate column chunks
// Every wait is bounded and raises the error word; the warps that wait together
// (2, 4..11) give up together.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "ffn_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace sgl {
namespace {

constexpr int kLinThreads = 384;
constexpr int kLinEpiWarp0 = 4, kLinEpiWarps = 8;
constexpr int kLinHalf = 128 * 128;         // one operand's stage: 128 rows of 128 bytes
constexpr int kLinStage = 2 * kLinHalf;     // A, B
constexpr int kLinTile = 256;               // features on M, columns on N
constexpr int kLinChunk = 768;      // most contraction per pass of an fp32 result
constexpr int kLinChunk16 = 16384;  // and of a bf16 result (wgrad; features end there)
constexpr int kLinCtrl = 512;
constexpr int kLinPitch = 80;               // a transposed row: 64 bytes, and 16 against conflicts
constexpr int kLinStages = 6;
constexpr int kLinBoxRow = 64;              // a stored box of wgrad: 32 rows of 64 bytes
constexpr int kLinBox = 32 * kLinBoxRow;

constexpr int kLinEpi = 32 * kLinPitch > kLinBox ? 32 * kLinPitch : kLinBox;  // per epilogue warp
constexpr int kLinSmem = kLinStages * kLinStage + kLinEpiWarps * kLinEpi + kLinCtrl + 1024 +
                         (2 * kMaxExpertsCfg + 2 + 33) * 4;
static_assert(kLinSmem <= 227 * 1024 && kLinEpi % 512 == 0, "shared memory");

struct LinParams {
  int E, R;
  int M, C;        // features on M; on N (wgrad only)
  int depth;       // contraction length (forward, dgrad)
  int mt;          // feature tiles on M
  long long ld;    // output row stride
  int out_f32, accumulate;
  const int32_t* offsets;
  void* out;
  int32_t* err;
  // test hooks of the waits: their limit in cycles, and arrivals added to those
  // that free an accumulator (some that never come make the waits run out)
  long long wait_limit;
  int ready_extra;
};

struct LinMaps {
  CUtensorMap a;       // forward: W, 128-row boxes; dgrad: W, wgrad: dy, 64-row boxes
  CUtensorMap b, b64, b32;  // forward, dgrad: rows, boxes of 128, 64, 32; wgrad: x, 64-row boxes
  CUtensorMap o;       // wgrad: dW, boxes of 32 rows of kLinBoxRow bytes
};

struct LinTile {
  int e, m0, c0;   // expert, first feature on M, first column (token row / feature)
  int rows, cols;  // rows of the contraction (wgrad) or of the tile; columns to store
  int n;           // MMA N: cols rounded up to 32
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Adds 16 bytes of fp32 to global memory without reading them back.
__device__ __forceinline__ void red_add_v4(float* p, const float4& v) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}

template <int DIR>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLinThreads, 1)
    grouped_linear(const __grid_constant__ LinParams p, const __grid_constant__ LinMaps m) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* epi = smem + kLinStages * kLinStage;
  uint8_t* ctrl = epi + kLinEpiWarps * kLinEpi;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);  // [stages] (the leader's count)
  uint64_t* empty = full + kLinStages;                 // [stages]
  uint64_t* tail = empty + kLinStages;                 // [stages] wgrad: a last block has landed
  uint64_t* tfull = tail + kLinStages;                 // [2]
  uint64_t* tempty = tfull + 2;                        // [2] (the leader's count)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* bad = const_cast<int*>(abort_flag) + 1;
  int* count = bad + 1;  // [2] column tiles of 256 and of 128
  static_assert(8 * (3 * kLinStages + 4) + 20 <= kLinCtrl, "ctrl");
  int* s_off = reinterpret_cast<int*>(ctrl + kLinCtrl);  // [E+1] row offsets
  int* s_tile = s_off + p.E + 1;                         // [E+1] tiles before expert e
  int* wsum = s_tile + p.E + 1;                          // [33]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank() & 1u;
  const bool leader = rank == 0;
  if (tid == 0) {
    for (int s = 0; s < kLinStages; ++s) {
      // the leader's producer; wgrad: two arrivals, its producer's or, for a
      // last block, one of each CTA's zeroing warp
      mbar_init(&full[s], DIR == kWgrad ? 2 : 1);
      mbar_init(&empty[s], 1);  // the leader's multicast commit
      mbar_init(&tail[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);  // multicast commit
      mbar_init(&tempty[a], 2 * kLinEpiWarps + p.ready_extra);  // the epilogue warps of both CTAs
    }
    *abort_flag = 0;
    *bad = count[0] = count[1] = 0;
    fence_mbar_init();
    if (p.R > 0) {
      prefetch_tmap(&m.a);
      prefetch_tmap(&m.b);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  pdl_wait();  // what follows reads and writes what earlier kernels wrote
  for (int i = tid; i <= p.E; i += kLinThreads) s_off[i] = p.offsets[i];
  tc_fence_before();
  __syncthreads();
  const int first = blockIdx.x / 2, pairs = gridDim.x / 2;
  int n256 = 0, n128 = 0;  // column tiles of this thread's experts
  for (int e = tid; e <= p.E; e += kLinThreads) {
    const int lo = s_off[e], hi = e < p.E ? s_off[e + 1] : p.R;
    if (lo < 0 || hi < lo || hi > p.R) {
      *bad = 1;
    } else if (e < p.E) {
      const int cols = DIR == kWgrad ? p.C : hi - lo;
      n256 += (cols + kLinTile - 1) / kLinTile;
      n128 += (cols + kLinTile / 2 - 1) / (kLinTile / 2);
    }
  }
  atomicAdd(&count[0], n256);
  atomicAdd(&count[1], n128);
  __syncthreads();
  const bool go = *bad == 0;  // the same in every CTA: all read the same offsets
  if (!go && tid == 0) atomicExch(p.err, MOE_DEVERR_OFFSETS);
  // Columns of a tile: 256, or 128 where so few tiles leave pairs idle in the
  // last of at most three rounds and the halves fill them (input gradient of 5003
  // rows, 32 experts of 200 x 1000: 21 us with 256, 17 with 128; weight gradient
  // of a single 768 x 2560 expert, 4096 rows: 28 and 22; 8 experts: 22 and 22).
  const int r256 = (count[0] * p.mt + pairs - 1) / pairs, r128 = (count[1] * p.mt + pairs - 1) / pairs;
  const int wide = r256 <= 3 && r128 < 2 * r256 ? kLinTile / 2 : kLinTile;
  const int ct = DIR == kWgrad ? (p.C + wide - 1) / wide : 0;  // column tiles of an expert
  if (go)
    for (int e = tid; e <= p.E; e += kLinThreads)
      s_tile[e] = e == p.E ? 0
                           : p.mt * (DIR == kWgrad ? ct : (s_off[e + 1] - s_off[e] + wide - 1) / wide);
  __syncthreads();
  if (go) smem_exscan(s_tile, p.E + 1, wsum);
  cluster_sync();  // both CTAs' barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int tiles = go ? s_tile[p.E] : 0;
  auto at_leader = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };

  // Tile i; e: the expert of the caller's previous tile (tiles ascend).
  auto tile_at = [&](int i, int e) {
    LinTile t;
    while (s_tile[e + 1] <= i) ++e;
    const int local = i - s_tile[e];
    const int rows = s_off[e + 1] - s_off[e];
    t.e = e;
    t.m0 = (local % p.mt) * kLinTile;
    const int c = (local / p.mt) * wide;
    if (DIR == kWgrad) {
      t.c0 = c;
      t.rows = rows;
      t.cols = min(wide, p.C - c);
    } else {
      t.c0 = s_off[e] + c;
      t.cols = t.rows = min(wide, rows - c);
    }
    t.n = (t.cols + 31) & ~31;
    return t;
  };
  // contraction per accumulator: equal shares, in whole 64-deep blocks
  auto chunk_of = [&](int depth) {
    const int most = p.out_f32 ? kLinChunk : kLinChunk16;
    if (depth <= most) return 1 << 30;
    const int blocks = (depth + 63) / 64, passes = (depth + most - 1) / most;
    return (blocks + passes - 1) / passes * 64;
  };
  // Passes of a bf16 result take one accumulator in turn; the other one holds
  // their sum, which only the epilogue touches. The next tile takes the first
  // one, too, so the MMAs are back at the sum's only when the epilogue has left it.
  auto summed = [&](int depth) { return DIR == kWgrad && !p.out_f32 && depth > kLinChunk16; };
  auto depth_of = [&](const LinTile& t) { return DIR == kWgrad ? t.rows : p.depth; };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (elect_one()) {
      const uint64_t pol = policy_evict_last(), pol_w = policy_evict_first();
      int stage = 0, e = 0;
      uint32_t phase = 0;
      bool live = true;
      for (int i = first; i < tiles && live; i += pairs) {
        const LinTile t = tile_at(i, e);
        e = t.e;
        const int depth = depth_of(t), half = t.n / 2;
        const int am = t.m0 + static_cast<int>(rank) * 128;
        const int bc = t.c0 + static_cast<int>(rank) * half;
        // B: 64-feature boxes (wgrad); of rows (forward, dgrad) one box of 128,
        // or one of 64 and one of 32, or either, the fewest that cover its half
        const int got = DIR == kWgrad ? (half + 63) & ~63 : half > 96 ? 128 : (half + 31) & ~31;
        const CUtensorMap* mb = got == 128 ? &m.b : got >= 64 ? &m.b64 : &m.b32;
        const uint32_t bytes = kLinHalf + got * 128;
        // weights that one tile column reads are not needed again
        const uint64_t pa = DIR != kWgrad && s_off[t.e + 1] - s_off[t.e] <= wide ? pol_w : pol;
        const int row0 = s_off[t.e];
        for (int k0 = 0; k0 < depth; k0 += 64) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.err, MOE_DEVERR_TIMEOUT, p.wait_limit)) {
            live = false;
            break;
          }
          uint8_t* sA = smem + stage * kLinStage;
          uint8_t* sB = sA + kLinHalf;
          if (DIR == kWgrad) {
            const int row = row0 + k0, rest = depth - k0;
            if (rest < 64 && rest % 16 != 0) {  // zeroed before it counts as full
              mbar_arrive_expect_tx(&tail[stage], bytes);
              for (int h = 0; h < 2; ++h)
                tma_load_2d(sA + h * 8192, &m.a, &tail[stage], am + 64 * h, row, pol);
              for (int h = 0; h < got / 64; ++h)
                tma_load_2d(sB + h * 8192, &m.b, &tail[stage], bc + 64 * h, row, pol);
            } else {
              const uint32_t bar = at_leader(&full[stage]);
              if (leader) {
                mbar_arrive(&full[stage]);
                mbar_arrive_expect_tx(&full[stage], 2 * bytes);
              }
              for (int h = 0; h < 2; ++h)
                tma_load_2d_pair(sA + h * 8192, &m.a, bar, am + 64 * h, row, pol);
              for (int h = 0; h < got / 64; ++h)
                tma_load_2d_pair(sB + h * 8192, &m.b, bar, bc + 64 * h, row, pol);
            }
          } else {
            const uint32_t bar = at_leader(&full[stage]);
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
            if (DIR == kFwd) {
              tma_load_3d_pair(sA, &m.a, bar, k0, am, t.e, pa);
            } else {
              for (int h = 0; h < 2; ++h)
                tma_load_3d_pair(sA + h * 8192, &m.a, bar, am + 64 * h, k0, t.e, pa);
            }
            tma_load_2d_pair(sB, mb, bar, k0, bc, pol);
            if (got == 96) tma_load_2d_pair(sB + 8192, &m.b32, bar, k0, bc + 64, pol);
          }
          if (++stage == kLinStages) stage = 0, phase ^= 1;
        }
      }
      // every stage must be released by the MMA before teardown
      for (int i = 0; i < kLinStages && live; ++i) {
        if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.err, MOE_DEVERR_TIMEOUT, p.wait_limit)) break;
        if (++stage == kLinStages) stage = 0, phase ^= 1;
      }
      // after a timeout: time for the copies and MMAs in flight to end (they take microseconds)
      if (*abort_flag)
        for (const long long t0 = clock64(); clock64() - t0 < 4000000;) {}
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (leader && elect_one()) {
      // The tensor pipe holds little more than one instruction, so whatever runs
      // between two blocks' MMAs shows: descriptors are additions to the stage's
      // first one, counters stand in for divisions, and the next tile is worked
      // out under this one's first MMAs.
      constexpr uint32_t major = DIR == kFwd ? 0 : DIR == kDgrad ? kIdescMnA : kIdescMnA | kIdescMnB;
      constexpr uint64_t step_a = (DIR == kFwd ? 32 : 2048) / 16, step_b = (DIR == kWgrad ? 2048 : 32) / 16;
      const uint32_t a0 = smem_u32(smem), b0 = a0 + kLinHalf;
      const uint64_t first_a = DIR == kFwd ? sdesc_k128(a0) : sdesc_mn128(a0, 8192);
      const uint64_t first_b = DIR == kWgrad ? sdesc_mn128(b0, 8192) : sdesc_k128(b0);
      uint64_t da = first_a, db = first_b;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t buf = 0, uses = 0;  // accumulator; bit b: parity of accumulator b's uses so far
      bool live = true;
      LinTile t;
      if (first < tiles) t = tile_at(first, 0);
      for (int i = first; i < tiles && live; i += pairs) {
        LinTile next = t;
        const int depth = depth_of(t);
        if (depth == 0) {
          if (i + pairs < tiles) t = tile_at(i + pairs, t.e);
          continue;
        }
        const uint32_t idesc = idesc_bf16(2 * 128, t.n) | major;
        const int chunk = chunk_of(depth);
        const uint32_t step = summed(depth) ? 0 : 1;  // to the next accumulator
        int left = 0;  // contraction left to this accumulator
        uint32_t d = 0;
        for (int rest = depth; rest > 0; rest -= 64) {
          const bool fresh = left <= 0;
          if (fresh) {  // the next accumulator
            if (rest < depth) umma_commit_pair_mc(&tfull[buf], 0x3), uses ^= 1u << buf, buf ^= step;
            if (!mbar_wait_cluster(&tempty[buf], ((uses >> buf) & 1) ^ 1, abort_flag, p.err,
                                   MOE_DEVERR_TIMEOUT, p.wait_limit)) {
              live = false;
              break;
            }
            d = tmem_base + buf * kLinTile;
            left = chunk;
          }
          left -= 64;
          if (!(DIR == kWgrad  // only there does the other CTA write what this one then reads
                    ? mbar_wait_cluster(&full[stage], phase, abort_flag, p.err, MOE_DEVERR_TIMEOUT, p.wait_limit)
                    : mbar_wait(&full[stage], phase, abort_flag, p.err, MOE_DEVERR_TIMEOUT, p.wait_limit))) {
            live = false;
            break;
          }
          tc_fence_after();
          if (rest > 48) {
            umma_bf16_pair(d, da, db, idesc, fresh ? 0u : 1u);
            umma_bf16_pair(d, da + step_a, db + step_b, idesc, 1u);
            umma_bf16_pair(d, da + 2 * step_a, db + 2 * step_b, idesc, 1u);
            umma_bf16_pair(d, da + 3 * step_a, db + 3 * step_b, idesc, 1u);
          } else {
            for (int k = 0; k < rest; k += 16)
              umma_bf16_pair(d, da + (k / 16) * step_a, db + (k / 16) * step_b, idesc,
                             fresh && k == 0 ? 0u : 1u);
          }
          umma_commit_pair_mc(&empty[stage], 0x3);  // frees the stage in both CTAs
          if (rest == depth && i + pairs < tiles) next = tile_at(i + pairs, t.e);
          da += kLinStage / 16, db += kLinStage / 16;
          if (++stage == kLinStages) stage = 0, phase ^= 1, da = first_a, db = first_b;
        }
        if (!live) break;
        umma_commit_pair_mc(&tfull[buf], 0x3), uses ^= 1u << buf, buf ^= step;
        t = next;
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ zeroing of ragged ends (wgrad)
    if (DIR == kWgrad) {
      int stage = 0, e = 0;
      uint32_t seen = 0;  // bit s: parity of stage s's tail barrier
      bool live = true;
      for (int i = first; i < tiles && live; i += pairs) {
        const LinTile t = tile_at(i, e);
        e = t.e;
        const int blocks = (t.rows + 63) / 64, rest = t.rows % 64;
        if (rest % 16 != 0) {
          const int s = (stage + blocks - 1) % kLinStages;
          if (!mbar_wait_warp(&tail[s], (seen >> s) & 1, abort_flag, p.err, MOE_DEVERR_TIMEOUT, p.wait_limit)) break;
          seen ^= 1u << s;
          // whole 128-byte rows: the swizzle moves pieces inside a row only
          uint8_t* base = smem + s * kLinStage;
          const int nrow = 16 - rest % 16;
          for (int j = lane; j < 4 * nrow * 8; j += 32) {
            const int box = j / (nrow * 8), row = rest + (j / 8) % nrow;
            *reinterpret_cast<uint4*>(base + box * 8192 + row * 128 + (j % 8) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (leader) mbar_arrive(&full[s]);
            else {
              fence_release_shared_cluster();
              mbar_arrive_cluster_relaxed(at_leader(&full[s]));
            }
          }
        }
        stage = (stage + blocks) % kLinStages;
      }
    }
  } else if (warp >= kLinEpiWarp0) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, part = (warp - kLinEpiWarp0) / 4;
    uint8_t* tile = epi + (warp - kLinEpiWarp0) * kLinEpi;
    int e = 0;
    uint32_t buf = 0, uses = 0;  // as in the MMA issuer
    const int box = kLinBoxRow / (p.out_f32 ? 4 : 2);  // columns of a stored box
    for (int i = first; i < tiles; i += pairs) {
      const LinTile t = tile_at(i, e);
      e = t.e;
      const int f0 = t.m0 + static_cast<int>(rank) * 128 + q * 32;  // this warp's features on M
      const int depth = depth_of(t);
      if (DIR == kWgrad && depth == 0) {
        // an expert without rows: this CTA's share of its matrix, which is one
        // stretch of memory, whatever the tile (tile by tile, the narrow ones at
        // its edges made this up to a third slower than writing products)
        if (p.accumulate) continue;
        const long long all = static_cast<long long>(p.M) * p.C * (p.out_f32 ? 4 : 2) / 16;
        const int shares = 2 * p.mt * ct;
        const int share = 2 * (t.c0 / wide * p.mt + t.m0 / kLinTile) + static_cast<int>(rank);
        uint4* o = static_cast<uint4*>(p.out) + t.e * all;
        const long long end = all * (share + 1) / shares;
        for (long long j = all * share / shares + (tid - kLinEpiWarp0 * 32); j < end; j += kLinEpiWarps * 32)
          o[j] = make_uint4(0, 0, 0, 0);
        continue;
      }
      const int chunk = chunk_of(depth);
      const bool sums = summed(depth);
      bool live = true;
      for (int k0 = 0; k0 == 0 || k0 < depth; k0 += chunk) {
        const bool add = p.accumulate || (k0 > 0 && !sums);
        if (!mbar_wait_warp(&tfull[buf], (uses >> buf) & 1, abort_flag, p.err, MOE_DEVERR_TIMEOUT, p.wait_limit)) {
          live = false;
          break;
        }
        tc_fence_after();
        // the pass before has reached the output (bulk stores keep no order)
        if (DIR == kWgrad && k0 > 0 && elect_one()) bulk_wait<0>();
        const uint32_t tq = tmem_base + buf * kLinTile + (static_cast<uint32_t>(q * 32) << 16);
        if (DIR == kWgrad) {
          // lane = row of D, whose columns are adjacent in dW: boxes of 32 rows
          // by TMA. The box ends at dW's edges by itself.
#pragma unroll 1
          for (int c0 = box * part; c0 < t.cols && f0 < p.M; c0 += 2 * box) {
            float v[32];
            tmem_ld16(tq + c0, v);
            if (!p.out_f32) tmem_ld16(tq + c0 + 16, v + 16);
            if (sums) {  // the sum of the passes, in the other accumulator
              tmem_ld_wait_for<32>(v);
              const uint32_t ts = tq + c0 + kLinTile - 2 * buf * kLinTile;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (k0 > 0) {
                  float w[16];
                  tmem_ld16(ts + 16 * h, w);
                  tmem_ld_wait_for<16>(w);
#pragma unroll
                  for (int j = 0; j < 16; ++j) v[16 * h + j] += w[j];
                }
                if (k0 + chunk < depth) tmem_st16(ts + 16 * h, v + 16 * h);
              }
              if (k0 + chunk < depth) continue;
            }
            if (elect_one()) bulk_wait_read<0>();  // the warp's box is free again
            __syncwarp();
            tmem_ld_wait_for<16>(v);
            if (!p.out_f32) tmem_ld_wait_for<16>(v + 16);
            auto put = [&](int piece, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
              const int at = piece ^ ((lane >> 1) & 3);  // the 64-byte swizzle
              *reinterpret_cast<uint4*>(tile + lane * kLinBoxRow + (at << 4)) = make_uint4(x, y, z, w);
            };
            if (p.out_f32) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                put(j, __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                    __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                put(j, pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                    pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (elect_one()) {
              if (add) tma_add_3d(&m.o, tile, t.c0 + c0, f0, t.e);
              else tma_store_3d(&m.o, tile, t.c0 + c0, f0, t.e);
              bulk_commit();
            }
          }
        } else {
          const int left = p.M - f0;  // features that exist
#pragma unroll 1
          for (int c0 = 32 * part; c0 < t.cols && left > 0; c0 += 64) {
            if (!p.out_f32) {
              // 32 features x 32 token rows, read as 8 x 8 fragments and stored
              // transposed: rows of 32 features
              float v[32];
              tmem_ld_16x32(tq + c0, v);
              tmem_ld_16x32(tq + (16u << 16) + c0, v + 16);
              tmem_ld_wait_for<32>(v);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float *lo = v + 4 * j, *hi = v + 16 + 4 * j;
                const uint32_t r[4] = {pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]),
                                       pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3])};
                stmatrix4_trans(tile + (8 * j + (lane & 7)) * kLinPitch + (lane >> 3) * 16, r);
              }
              __syncwarp();
              const int piece = lane & 3;
              uint16_t* o = static_cast<uint16_t*>(p.out) + (t.c0 + c0 + lane / 4) * p.ld + f0 + piece * 8;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = lane / 4 + 8 * j;
                if (c0 + r < t.cols && piece * 8 < left)
                  *reinterpret_cast<uint4*>(o + 8 * j * p.ld) =
                      *reinterpret_cast<const uint4*>(tile + r * kLinPitch + piece * 16);
              }
              __syncwarp();
            } else {
              // lane = feature: 16 token rows at a time, rows of 128 bytes, 144 apart
              float v[32];
              tmem_ld16(tq + c0, v);
              tmem_ld16(tq + c0 + 16, v + 16);
              tmem_ld_wait_for<32>(v);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  *reinterpret_cast<float*>(tile + j * 144 + lane * 4) = v[16 * h + j];
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int r = lane / 8 + 4 * j, c = (lane & 7) * 4;
                  const int tok = c0 + 16 * h + r;
                  if (tok < t.cols && c < left) {
                    const float4 x = *reinterpret_cast<const float4*>(tile + r * 144 + c * 4);
                    float* o = static_cast<float*>(p.out) + (t.c0 + tok) * p.ld + f0 + c;
                    if (add) red_add_v4(o, x);
                    else *reinterpret_cast<float4*>(o) = x;
                  }
                }
                __syncwarp();
              }
            }
          }
        }
        if (sums) tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // hands over tensor memory only, which the tcgen05 fence orders; a release
          // at cluster scope would wait for this tile's global stores
          if (leader) mbar_arrive(&tempty[buf]);
          else mbar_arrive_cluster_relaxed(at_leader(&tempty[buf]));
        }
        uses ^= 1u << buf;
        if (!sums) buf ^= 1;
      }
      if (!live) break;
    }
    if (DIR == kWgrad) {
      __syncwarp();
      if (elect_one()) bulk_wait<0>();
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while the other may still arrive on its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// CTA pairs that the device runs at once (a pair's two SMs lie in one cluster
// of SMs, so this may be less than half the SMs); cached per device.
template <int DIR>
cudaError_t resident_pairs(int smem, int* pairs) {
  static int cache[kMaxDevices] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (cache[dev] == 0) {
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof(lc));
    lc.gridDim = dim3(num_sms() & ~1);
    lc.blockDim = dim3(kLinThreads);
    lc.dynamicSmemBytes = smem;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, grouped_linear<DIR>, &lc);
    if (e != cudaSuccess) return e;
    cache[dev] = n < 1 ? 1 : n;
  }
  *pairs = cache[dev];
  return cudaSuccess;
}

template <int DIR>
cudaError_t run(const moe_linear_desc& d, LinParams p, const LinMaps& m, cudaStream_t s) {
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(grouped_linear<DIR>), kLinSmem);
  if (e != cudaSuccess) return e;
  int pairs = 0;
  if ((e = resident_pairs<DIR>(kLinSmem, &pairs)) != cudaSuccess) return e;
  // no more pairs than tiles there can be
  const long long most = DIR == kWgrad
                             ? 1LL * d.E * p.mt * cdiv(p.C, kLinTile / 2)
                             : 1LL * p.mt * (cdiv(d.R, kLinTile / 2) + (d.E < d.R ? d.E : d.R));
  if (most < pairs) pairs = static_cast<int>(most);
  return launch_pdl(grouped_linear<DIR>, dim3(2 * pairs), dim3(kLinThreads), kLinSmem, s, p, m);
}

}  // namespace

cudaError_t launch_grouped_linear(const moe_linear_desc& d, LinearDir dir, const void* a,
                                  const void* b, const int32_t* offsets, void* out, int32_t* err,
                                  cudaStream_t s) {
  // A few rows, spread over the experts: bound by the weights of rows that share
  // none, see linear_few.cu. Calls back to back in a graph, weights not in L2, there
  // and here, us:
  //   rows                          8           16           32           64           128
  //   768 x 2560, an expert each  9.5, 28.6  14.7, 29.9  25.0, 51.2  44.2, 65.2  82.6, 101.5
  //   2560 x 768, an expert each  9.0, 37.6  14.0, 42.8  24.2, 50.3  42.4, 63.3  80.4,  91.2
  //   768 x 2560, one expert      6.7, 13.4  11.2, 13.4    - , 13.5    - , 13.7    - ,  14.6
  //   2560 x 768, one expert      6.7,  8.2  10.6,  8.2    - ,  8.3    - ,  8.5    - ,   9.1
  // R is the rows' capacity: the live rows are known on the device only.
  if (dir == kFwd && d.R <= kFewMaxRows && (d.R <= 16 || d.R <= 4 * d.E))
    return launch_linear_few(d, a, b, offsets, out, err, s);
  LinParams p;
  memset(&p, 0, sizeof(p));
  p.E = d.E;
  p.R = d.R;
  p.M = dir == kDgrad ? d.K : d.N;
  p.C = dir == kWgrad ? d.K : 0;
  p.depth = dir == kFwd ? d.K : d.N;
  p.mt = cdiv(p.M, kLinTile);
  p.ld = dir == kFwd ? d.ld_y : dir == kDgrad ? d.ld_x : d.K;
  p.out_f32 = d.out_type == MOE_T_F32;
  p.accumulate = d.accumulate != 0;
  p.offsets = offsets;
  p.out = out;
  p.err = err;
  p.wait_limit = kWaitLimitCycles;
  if (const char* v = getenv("SGL_MOE_TEST_WAIT_CYCLES")) p.wait_limit = strtoll(v, nullptr, 10);
  if (const char* v = getenv("SGL_MOE_TEST_READY_EXTRA"))
    p.ready_extra = static_cast<int>(max(0L, min(1000L, strtol(v, nullptr, 10))));
  LinMaps m;
  memset(&m, 0, sizeof(m));
  bool ok = true;
  if (dir == kWgrad) {
    // no rows: every tile is empty and no map is read
    ok = map_store_blocks(&m.o, out, p.out_f32 != 0, d.E, d.N, d.K, 32, kLinBoxRow);
    if (d.R > 0)
      ok = ok && map_bf16_ld(&m.a, a, d.R, d.N, d.ld_y, 64) && map_bf16_ld(&m.b, b, d.R, d.K, d.ld_x, 64);
  } else {
    const int width = dir == kFwd ? d.K : d.N, ld = dir == kFwd ? d.ld_x : d.ld_y;
    ok = map_bf16_blocks(&m.a, b, d.E, d.N, d.K, dir == kFwd ? 128 : 64) &&
         map_bf16_ld(&m.b, a, d.R, width, ld, 128) && map_bf16_ld(&m.b64, a, d.R, width, ld, 64) &&
         map_bf16_ld(&m.b32, a, d.R, width, ld, 32);
  }
  if (!ok) return cudaErrorInvalidValue;
  switch (dir) {
    case kFwd: return run<kFwd>(d, p, m, s);
    case kDgrad: return run<kDgrad>(d, p, m, s);
    default: return run<kWgrad>(d, p, m, s);
  }
}

}  // namespace sgl
