// expert_fp8.cu -- the expert layer on 8-bit operands: the layer of
// expert_ffn.cu with weights and activations in E4M3 and fp32 scales.
//
// "Kolibri 1 im Detail", FP8 section: weights in E4M3 with one fp32 scale per
// 128 x 128 block, activations with one per 1 x 128 group; the router stays
// bf16.  For slot p of expert e and token t:
//   g, u  = sum over k blocks b of  xs[t,b] ws[e,.,b] (sum_{k in b} x8 w8)    fp32
//   h     = SiLU(g) u, then per 128 units hs = max(amax|h|, 1e-30) / 448, h8 = e4m3(h / hs)
//   o[p]  = sum over unit blocks b of  hs[p,b] wds[e,.,b] (sum h8 wd8)        fp32, rounded to bf16
//   y[t]  = o_shared[t] + sum_k gates[t,k] o[inv[t K + k]]                    fp32, rounded to bf16
//
// The scales are arbitrary fp32 numbers per 128 values of k, so the tensor
// cores' block scaling (powers of two per 32) does not apply: each 128-wide k
// block is multiplied into its own TMEM buffer (kind::f8f6f4, four MMAs of K =
// 32, M = 128 token rows, N = 256 weight rows) and eight warps add it, scaled,
// to fp32 sums in registers while the next block is multiplied into the other
// buffer.  Token rows are the M side: a thread then owns one row, whose scale
// is one register, and the 1 x 128 group maximum of h is a maximum over the
// thread's own values and its partner's.
//
// The token rows are gathered by the TMA unit (tile::gather4) straight from
// x8, so there is no dispatch pass.  The shared expert is one more group of
// the same launch.  o is kept in bf16 (one rounding of 2^-9 per expert output,
// below the 2^-9 of y itself once summed): it is written and read once, N K d
// values, and would otherwise be the largest traffic of the layer.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "launch.h"
#include "gemm_pair.cuh"
#include "pdl.cuh"

namespace kolibri {

namespace {

using namespace gemm;

constexpr int kTokRows = 128;            // token rows of a tile: the MMA's M
constexpr int kWRows = 256;              // weight rows of a tile: the MMA's N
constexpr int kKBlock = 128;             // k values per scale: one 128-byte swizzle row
constexpr int kF8Stages = 4;
constexpr uint32_t kABytes = kTokRows * kKBlock;            // 16 KB
constexpr uint32_t kBBytes = kWRows * kKBlock;              // 32 KB
constexpr uint32_t kF8Stage = kABytes + kBBytes;
constexpr int kSumWarps = 8;
constexpr int kF8Threads = 64 + 32 * kSumWarps;             // warp 0 TMA, warp 1 MMA, warps 2..9 sums
constexpr int kF8Groups = KOLIBRI_MAX_EXPERTS + 1;          // the experts and the shared expert
constexpr float kF8AmaxMin = 1e-30f;
constexpr float kF8Max = 448.0f;

struct Fp8Params {
  const int64_t* offsets;   // [E + 1]
  const int32_t* perm;      // [N K]; gate/up only
  const float* a_scale;     // gate/up: [N, k_blocks] by token; down: [rows, k_blocks] by grouped row
  const float* w_scale;     // [E, w_rows / 128, k_blocks]
  const float* ws_scale;    // the shared expert's, or null
  void* out;                // gate/up: h8 [rows, F]; down: o [rows, d] bf16
  float* out_scale;         // gate/up: hs [rows, F / 128]
  int64_t N, NK;
  int K, E, shared;
  int k_blocks, n_tiles, ncols, w_rows;
};

struct F8Bars {
  uint32_t base;
  __device__ __forceinline__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return base + 8u * (kF8Stages + s); }
  __device__ __forceinline__ uint32_t tfull(int a) const { return base + 8u * (2 * kF8Stages + a); }
  __device__ __forceinline__ uint32_t tempty(int a) const { return base + 8u * (2 * kF8Stages + 2 + a); }
  __device__ __forceinline__ uint32_t holder() const { return base + 8u * (2 * kF8Stages + 4); }
};
constexpr int kF8BarBytes = 8 * (2 * kF8Stages + 5);

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

// Four rows of the map (box one row high), c0 .. c0 + 127 of each, to 512 bytes at dst.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int c0, int4 rows, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar),
      "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: D fp32, A and B E4M3, both K-major.
constexpr uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// SiLU(g) u by the fast exponential and division: a few fp32 units, far below the step of e4m3.
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// All threads: mt[g] = token blocks of the groups before g (mt[G] all of
// them) and off[g] = first grouped row of g; the shared expert is group E with
// rows [NK, NK + N).  Offsets that do not run from 0 to NK without decreasing
// are flagged and give no tiles.
__device__ void f8_tile_prefix(const Fp8Params& p, int G, int32_t* mt, int64_t* off, int32_t* warp_tot) {
  __shared__ int bad_s;
  if (threadIdx.x == 0) bad_s = 0;
  __syncthreads();
  for (int g = threadIdx.x; g <= p.E; g += kF8Threads) {
    const int64_t o = p.offsets[g];
    off[g] = o;
    const bool ok = (g > 0 || o == 0) && (g < p.E || o == p.NK) && o <= p.NK && (g == 0 || p.offsets[g - 1] <= o);
    if (!ok) bad_s = 1;
  }
  if (threadIdx.x == 0) off[p.E + 1] = p.NK + p.N;
  __syncthreads();
  const bool bad = bad_s != 0;
  if (bad && threadIdx.x == 0 && blockIdx.x == 0) raise_status(kStatusBadInput);
  constexpr int kPer = (kF8Groups + 1 + kF8Threads - 1) / kF8Threads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t v[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = tid * kPer + i;
    v[i] = g < G && !bad ? static_cast<int32_t>((off[g + 1] - off[g] + kTokRows - 1) / kTokRows) : 0;
    sum += v[i];
  }
  int32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  int32_t run = incl - sum;
  for (int w = 0; w < warp; ++w) run += warp_tot[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int g = tid * kPer + i;
    if (g <= G) mt[g] = run;
    run += v[i];
  }
  __syncthreads();
}

struct F8Tiles {
  const int32_t* mt;
  const int64_t* off;
  int G, n_tiles;
  // tile -> group, first grouped row, rows of the tile that exist, feature block
  __device__ __forceinline__ void map(int64_t tile, int& g, int64_t& row0, int& valid, int& n) const {
    const int mb = static_cast<int>(tile / n_tiles);
    n = static_cast<int>(tile - static_cast<int64_t>(mb) * n_tiles);
    int lo = 0, hi = G - 1;                   // last g with mt[g] <= mb
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (mt[mid] <= mb) lo = mid;
      else hi = mid - 1;
    }
    g = lo;
    row0 = off[g] + static_cast<int64_t>(mb - mt[g]) * kTokRows;
    const int64_t left = off[g + 1] - row0;
    valid = static_cast<int>(left < kTokRows ? left : kTokRows);
  }
};

// The token of grouped row `row`; N (out of range, read as zeros) for a bad entry.
__device__ __forceinline__ int64_t token_of(const Fp8Params& p, int64_t row) {
  if (row >= p.NK) return row - p.NK;
  const int32_t j = __ldg(p.perm + row);
  if (j < 0 || j >= p.NK) {
    raise_status(kStatusBadInput);
    return p.N;
  }
  return j / p.K;
}

template <bool kGateUp>
__global__ void __launch_bounds__(kF8Threads, 1)
    expert_fp8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_ws, const Fp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int32_t mt_s[kF8Groups + 1];
  __shared__ int64_t off_s[kF8Groups + 1];
  __shared__ int32_t warp_tot[kF8Threads / 32];
  __shared__ float amax_s[2][kTokRows];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  const F8Bars bars{ring + kF8Stage * kF8Stages};
  uint8_t* const holder_ptr = smem_raw + (bars.holder() - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.E + p.shared;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kF8Stages; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bars.tfull(a), 1);
      mbar_init(bars.tempty(a), kSumWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(bars.holder()) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  f8_tile_prefix(p, G, mt_s, off_s, warp_tot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(holder_ptr);
  const F8Tiles tiles{mt_s, off_s, G, p.n_tiles};
  const int64_t total = static_cast<int64_t>(mt_s[G]) * p.n_tiles;

  if (warp == 0) {
    // TMA producer: lane l gathers rows 4l .. 4l + 3 of the tile (gate/up); lane 0 loads the weights
    const uint64_t pol_w = policy_evict_first();
    const uint64_t pol_a = policy_evict_last();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      int g, valid, n;
      int64_t row0;
      tiles.map(tile, g, row0, valid, n);
      const bool sh = g == p.E;
      const CUtensorMap* tw = sh ? &tm_ws : &tm_w;
      const int w0 = (sh ? 0 : g * p.w_rows) + n * (kGateUp ? 128 : 256);
      const int w1 = w0 + (kGateUp ? p.w_rows / 2 : 128);
      int4 rows = make_int4(0, 0, 0, 0);
      const bool mine = kGateUp ? 4 * lane < valid : (lane < 4 && 32 * lane < valid);
      if (kGateUp && mine) {
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          r[i] = 4 * lane + i < valid ? static_cast<int>(token_of(p, row0 + 4 * lane + i)) : static_cast<int>(p.N);
        rows = make_int4(r[0], r[1], r[2], r[3]);
      }
      const uint32_t bytes = kBBytes + (kGateUp ? 512u * ((valid + 3) / 4) : 4096u * ((valid + 31) / 32));
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        if (!mbar_wait(bars.empty(stage), phase ^ 1u)) { ok = false; break; }
        const uint32_t a_dst = ring + kF8Stage * stage, b_dst = a_dst + kABytes;
        if (lane == 0) {
          mbar_arrive_expect_tx(bars.full(stage), bytes);
          tma_load_2d(b_dst, tw, kb * kKBlock, w0, bars.full(stage), pol_w);
          tma_load_2d(b_dst + kBBytes / 2, tw, kb * kKBlock, w1, bars.full(stage), pol_w);
        }
        __syncwarp();
        if (mine) {
          if constexpr (kGateUp) tma_gather4(a_dst + 512u * lane, &tm_a, kb * kKBlock, rows, bars.full(stage), pol_a);
          else tma_load_2d(a_dst + 4096u * lane, &tm_a, kb * kKBlock, static_cast<int>(row0) + 32 * lane, bars.full(stage), pol_a);
        }
        if (++stage == kF8Stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc_e4m3(kTokRows, kWRows);
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(bars.tempty(buf), buf_phase ^ 1u) || !mbar_wait(bars.full(stage), phase)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = ring + kF8Stage * stage;
          const uint64_t a_desc = sw128_desc(a_addr), b_desc = sw128_desc(a_addr + kABytes);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)       // 32 e4m3 along k = 32 bytes inside the swizzle row
            tc_mma_f8(tmem_base + 256u * buf, a_desc + 2u * ks, b_desc + 2u * ks, idesc, ks > 0 ? 1u : 0u);
          tc_commit(bars.empty(stage));
          tc_commit(bars.tfull(buf));
          if (++stage == kF8Stages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == 2) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
    }
  } else {
    // sums: thread = token row (TMEM lane quarter warp % 4), half of the columns.
    // Gate/up: half h holds the gates and the ups of units 64 h .. 64 h + 63.
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    int buf = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    for (int64_t tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      int g, valid, n;
      int64_t row0;
      tiles.map(tile, g, row0, valid, n);
      const bool sh = g == p.E;
      const bool live = r < valid, warp_live = quarter * 32 < valid;
      const int64_t row = row0 + r;
      int64_t arow = row;
      if (kGateUp && live) arow = token_of(p, row);
      const bool have = live && (!kGateUp || arow < p.N);
      const float* as = p.a_scale + arow * p.k_blocks;
      const int wblocks = p.w_rows / 128;
      const float* wbase = sh ? p.ws_scale : p.w_scale + static_cast<int64_t>(g) * wblocks * p.k_blocks;
      const float* w0 = wbase + (kGateUp ? n : 2 * n + half) * p.k_blocks;
      const float* w1 = kGateUp ? w0 + (wblocks / 2) * p.k_blocks : w0;
      float acc[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c][i] = 0.0f;
      float sa = have ? __ldg(as) : 0.0f, s0 = __ldg(w0), s1 = __ldg(w1);
      for (int kb = 0; kb < p.k_blocks; ++kb) {
        const float f0 = sa * s0, f1 = sa * s1;
        if (kb + 1 < p.k_blocks) {
          sa = have ? __ldg(as + kb + 1) : 0.0f;
          s0 = __ldg(w0 + kb + 1);
          s1 = __ldg(w1 + kb + 1);
        }
        if (!mbar_wait(bars.tfull(buf), buf_phase)) { ok = false; break; }
        tc_fence_after();
        if (warp_live) {
          const uint32_t t0 = tmem_base + lane_off + 256u * buf + (kGateUp ? 64u : 128u) * half;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(t0 + (kGateUp && c >= 2 ? 64u : 0u) + 32u * c, v);
            tmem_wait_ld();
            const float f = c < 2 ? f0 : f1;
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c][i] = fmaf(__uint_as_float(v[i]), f, acc[c][i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.tempty(buf));
        if (++buf == 2) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      if (!ok) break;
      if constexpr (kGateUp) {
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            acc[c][i] = silu_mul(acc[c][i], acc[c + 2][i]);
            amax = fmaxf(amax, fabsf(acc[c][i]));
          }
        amax_s[half][r] = amax;
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kSumWarps) : "memory");
        amax = fmaxf(fmaxf(amax, amax_s[half ^ 1][r]), kF8AmaxMin);
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kSumWarps) : "memory");
        if (live) {
          const float q = __fdiv_rn(kF8Max, amax);
          uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + row * p.ncols + n * 128 + half * 64);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* a = &acc[j >> 1][(j & 1) * 16];
            o[j] = make_uint4(pack_e4m3(a[0] * q, a[1] * q, a[2] * q, a[3] * q),
                              pack_e4m3(a[4] * q, a[5] * q, a[6] * q, a[7] * q),
                              pack_e4m3(a[8] * q, a[9] * q, a[10] * q, a[11] * q),
                              pack_e4m3(a[12] * q, a[13] * q, a[14] * q, a[15] * q));
          }
          if (half == 0) p.out_scale[row * p.n_tiles + n] = __fdiv_rn(amax, kF8Max);
        }
      } else if (live) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + row * p.ncols + n * 256 + half * 128);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float* a = &acc[j >> 2][(j & 3) * 8];
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(a[2 * i], a[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          o[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
}

// y[t] = o[NK + t] (shared) + sum_k gates[t,k] o[inv[t K + k]], fp32
// multiply-adds in the order shared, k ascending; eight columns per thread.
constexpr int kMaxCombineK = 16;
__global__ void __launch_bounds__(256) combine_fp8_kernel(const uint4* __restrict__ o, const int32_t* __restrict__ inv,
                                                          const float* __restrict__ gates, int64_t N, int K, int64_t NK,
                                                          int shared, int vecs, uint4* __restrict__ y) {
  __shared__ int64_t slot[kMaxCombineK + 1];
  __shared__ float gate[kMaxCombineK + 1];
  pdl_wait();
  for (int64_t t = blockIdx.x; t < N; t += gridDim.x) {
    __syncthreads();
    if (threadIdx.x < K) {
      const int32_t q = __ldg(inv + t * K + threadIdx.x);
      const bool ok = q >= 0 && q < NK;
      if (!ok) raise_status(kStatusBadInput);
      slot[threadIdx.x + shared] = ok ? q : -1;
      gate[threadIdx.x + shared] = __ldg(gates + t * K + threadIdx.x);
    }
    if (shared && threadIdx.x == 0) {
      slot[0] = NK + t;
      gate[0] = 1.0f;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
      float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int k = 0; k < K + shared; ++k) {
        if (slot[k] < 0) continue;
        const float s = gate[k];
        const uint4 v = __ldg(o + slot[k] * vecs + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[2 * i] = __fmaf_rn(s, __uint_as_float(w[i] << 16), a[2 * i]);
          a[2 * i + 1] = __fmaf_rn(s, __uint_as_float(w[i] & 0xffff0000u), a[2 * i + 1]);
        }
      }
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(a[2 * i], a[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      y[t * vecs + c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <bool kGateUp>
cudaError_t launch_fp8_gemm(const void* a, int64_t a_rows, const void* w, const void* w_shared, const Fp8Params& p,
                            cudaStream_t s) {
  const uint64_t kdim = static_cast<uint64_t>(p.k_blocks) * kKBlock;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap tm_a, tm_w, tm_ws;
  if (!encode_2d(&tm_a, u8, 1, a, kdim, static_cast<uint64_t>(a_rows), kKBlock, kGateUp ? 1 : 32) ||
      !encode_2d(&tm_w, u8, 1, w, kdim, static_cast<uint64_t>(p.E) * p.w_rows, kKBlock, 128) ||
      !encode_2d(&tm_ws, u8, 1, w_shared ? w_shared : w, kdim, static_cast<uint64_t>(p.w_rows), kKBlock, 128))
    return cudaErrorInvalidValue;
  auto kern = expert_fp8_kernel<kGateUp>;
  const size_t smem = 1024 + static_cast<size_t>(kF8Stage) * kF8Stages + kF8BarBytes;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  // token blocks: at most one partial block per group that has rows
  const int64_t rows = p.NK + (p.shared ? p.N : 0);
  const int64_t partial = p.NK < p.E ? p.NK : p.E;
  const int64_t tiles = (rows / kTokRows + partial + p.shared) * p.n_tiles;
  const int64_t sms = device_sm_count();
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(kF8Threads), smem, s,
                    dim3(0, 0, 0), tm_a, tm_w, tm_ws, p);
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Fp8Layout {
  size_t off_h8, off_hs, off_o, total;
};
Fp8Layout fp8_layout(int64_t N, int32_t d, int32_t F, int32_t K, bool shared) {
  const size_t rows = static_cast<size_t>(N) * K + (shared ? N : 0);
  Fp8Layout L{};
  L.off_h8 = 0;
  L.off_hs = up256(rows * F);
  L.off_o = L.off_hs + up256(rows * (F / 128) * sizeof(float));
  L.total = L.off_o + up256(rows * d * sizeof(uint16_t));
  return L;
}

}  // namespace

bool expert_fp8_shape_supported(int32_t d, int32_t F, int32_t E) {
  return d >= 256 && d % 256 == 0 && d <= 8192 && F >= 128 && F % 128 == 0 && F <= 8192 && E >= 1 &&
         E <= KOLIBRI_MAX_EXPERTS && static_cast<int64_t>(E) * 2 * F < (1LL << 31) &&
         static_cast<int64_t>(E) * d < (1LL << 31);
}

size_t expert_fp8_ws_bytes(int64_t N, int32_t d, int32_t F, int32_t K, bool shared) {
  return fp8_layout(N, d, F, K, shared).total;
}

cudaError_t launch_expert_ffn_fp8(const ExpertFp8Args& a, cudaStream_t s) {
  const bool shared = a.ws_gate_up != nullptr;
  const Fp8Layout L = fp8_layout(a.N, a.d, a.F, a.K, shared);
  char* base = static_cast<char*>(a.ws);
  const int64_t NK = a.N * a.K, rows = NK + (shared ? a.N : 0);
  Fp8Params p{};
  p.offsets = a.offsets;
  p.N = a.N;
  p.NK = NK;
  p.K = a.K;
  p.E = a.E;
  p.shared = shared ? 1 : 0;
  p.perm = a.perm;
  p.a_scale = a.x_scale;
  p.w_scale = a.s_gate_up;
  p.ws_scale = a.ss_gate_up;
  p.out = base + L.off_h8;
  p.out_scale = reinterpret_cast<float*>(base + L.off_hs);
  p.k_blocks = a.d / 128;
  p.n_tiles = a.F / 128;
  p.ncols = a.F;
  p.w_rows = 2 * a.F;
  cudaError_t err = launch_fp8_gemm<true>(a.x8, a.N, a.w_gate_up, a.ws_gate_up, p, s);
  if (err != cudaSuccess) return err;
  p.a_scale = reinterpret_cast<const float*>(base + L.off_hs);
  p.w_scale = a.s_down;
  p.ws_scale = a.ss_down;
  p.out = base + L.off_o;
  p.out_scale = nullptr;
  p.k_blocks = a.F / 128;
  p.n_tiles = a.d / 256;
  p.ncols = a.d;
  p.w_rows = a.d;
  err = launch_fp8_gemm<false>(base + L.off_h8, rows, a.w_down, a.ws_down, p, s);
  if (err != cudaSuccess) return err;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 8;
  return launch_pdl(combine_fp8_kernel, dim3(static_cast<unsigned>(a.N < cap ? a.N : cap)), dim3(256), 0, s,
                    dim3(0, 0, 0), reinterpret_cast<const uint4*>(base + L.off_o), a.inv, a.gates, a.N, a.K, NK,
                    shared ? 1 : 0, a.d / 8, static_cast<uint4*>(a.y));
}

KOLIBRI_DEFINE_STATUS_TAKE(status_take_expert_fp8)

}  // namespace kolibri
