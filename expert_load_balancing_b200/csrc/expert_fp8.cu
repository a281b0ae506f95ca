// expert_fp8.cu -- the expert layer on 8-bit operands: the layer of
// expert_ffn.cu with weights and activations in E4M3 and fp32 scales.
//
// "Kolibri 1 im Detail", FP8 section: weights in E4M3 with one fp32 scale per
// 128 x 128 block, activations with one per 1 x 128 group; the router stays
// bf16.  For slot p of expert e and token t:
//   g, u  = sum over k blocks b of  xs[t,b] ws[e,.,b] (sum_{k in b} x8 w8)    fp32
//   h     = SiLU(g) u, then per 128 units hs = max(amax|h|, 1e-30) / 448, h8 = e4m3(h 448 / max(amax|h|, 1e-30))
//   o[p]  = sum over unit blocks b of  hs[p,b] wds[e,.,b] (sum h8 wd8)        fp32, kept in fp16 (below)
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
// A first pass copies the token rows to their grouped places and lays their
// scales out by k block.  Gathering in the kernel was slower: by the TMA
// unit's row gather (four rows per instruction) the loads alone took 108 us
// where tiled loads take 55 (2049 tokens, 128 experts), and by cp.async, whose
// requests queue behind the bulk loads, the projection took 1615 us instead of
// 514 (16384 tokens, 384 experts).  The shared expert is one more group of the
// same launch.  o is kept in fp16 with a power of two per 1 x 128 group, which
// costs each value one rounding of at most 2^-11 of itself (an eighth of y's own
// to bf16; values below 2^-28 of the group's largest lose more): it is written
// and read once, N K d values, and in fp32 would be the largest traffic of the
// layer.
//
// Measured (d = 2560, F = 512, 6 of 384 experts and the shared one): 16384 tokens
// 873-890 us in a burst (gather 65, gate/up 412, down 282, combine 113), 1040 in
// a loop of seconds, where the power limit takes the clock to 1.53 GHz.  What
// bounds the two products is the SM's shared memory and tensor pipe in turn: loads
// alone take 266 and 208 us, loads and MMAs 340 and 258, MMAs alone 205 and 161,
// the sums alone 289 and 204.  64 tokens 172 us, bound by the weights' 0.95 GB.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "launch.h"
#include "approx.cuh"
#include "gemm_pair.cuh"
#include "pdl.cuh"

namespace kolibri {

namespace {

using namespace gemm;

constexpr int kTokRows = 128;            // token rows of a tile: the MMA's M
constexpr int kWRows = 256;              // weight rows of a tile: the MMA's N
constexpr int kKBlock = 128;             // k values per scale: one 128-byte swizzle row
constexpr int kMaxF8Stages = 4;
constexpr uint32_t kABytes = kTokRows * kKBlock;            // 16 KB
constexpr uint32_t kBBytes = kWRows * kKBlock;              // 32 KB
constexpr uint32_t kF8Stage = kABytes + kBBytes;
constexpr int kSumWarps = 8;
constexpr int kF8Threads = 128 + 32 * kSumWarps;            // warp 0 TMA, warps 1, 2 MMA, warp 3 tiles, warps 4..11 sums
// Register split: a launch of 384 threads has 168 each, 64,512 in all; the
// first warpgroup keeps 56 and the two summing ones take 224 (128 sums and two
// 32-column loads): 128 * 56 + 256 * 224 = 64,512.
constexpr int kF8RegsLow = 56, kF8RegsSum = 224;
constexpr int kF8Groups = KOLIBRI_MAX_EXPERTS + 1;          // the experts and the shared expert
constexpr float kF8AmaxMin = 1e-30f;
constexpr float kF8Max = 448.0f;

struct Fp8Params {
  const int64_t* offsets;   // [E + 1]
  const float* w_scale;     // [E, w_rows / 128, k_blocks]
  const float* ws_scale;    // the shared expert's, or null
  void* out;                // gate/up: h8 [rows, F]; down: o [rows, d] fp16
  float* out_scale;         // gate/up: hs [F / 128][ld]; down: [rows, d / 128]
  int64_t N, NK;
  int64_t ld;               // row length of the transposed scales
  int E, shared;
  int k_blocks, n_tiles, ncols, w_rows;
};

// full(s): the operands of stage s are there.  done(s): the MMAs on stage s are
// complete, which frees the stage and hands the buffer to the sums.  free(b):
// the sums have read TMEM buffer b.  tile(t), told(t): slot t holds the next
// tile's place and weight scales, the sums are through with them.
struct F8Bars {
  uint32_t base;
  __device__ __forceinline__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ __forceinline__ uint32_t done(int s) const { return base + 8u * (kMaxF8Stages + s); }
  __device__ __forceinline__ uint32_t free(int b) const { return base + 8u * (2 * kMaxF8Stages + b); }
  __device__ __forceinline__ uint32_t tile(int t) const { return base + 8u * (2 * kMaxF8Stages + 2 + t); }
  __device__ __forceinline__ uint32_t told(int t) const { return base + 8u * (2 * kMaxF8Stages + 4 + t); }
  __device__ __forceinline__ uint32_t holder() const { return base + 8u * (2 * kMaxF8Stages + 6); }
};
constexpr int kF8BarBytes = (8 * (2 * kMaxF8Stages + 7) + 15) / 16 * 16;
// Output rows pass through shared memory.  h8 (16 KB a tile): 64 bytes of 32
// rows per summing warp, written by neighbouring lanes as whole sectors (a store
// takes a cycle for each line that it touches); 80 bytes from row to row keep
// both ways free of bank conflicts.  o (64 KB a tile): a warp's 32 rows of 128
// columns as two 128-byte wide boxes that the TMA unit stores behind the next
// tile's sums; stored by the warps they held the sums up for 2 us a tile (385
// us instead of 235 without stores, 16384 tokens).  The down projection pays
// for that buffer with a stage, of which it needs fewer.
template <bool kGateUp>
struct F8Cfg {
  static constexpr int kStages = kGateUp ? 4 : 3;
  static constexpr int kOutPitch = 80;
  static constexpr int kOutBytes = kGateUp ? 32 * kOutPitch : 2 * 32 * 128;
};
// Row scales ride with the operands: the scales of a k block lie side by side
// by row, and one TMA copy brings the tile's (132 from the 16-byte boundary at
// or below its first row) into one of six slots.  A slot is overwritten six
// blocks later, when the MMAs of block + 2 (or + 3) are done, which wait for the
// sums of this block: no barrier of its own.  Loaded by the summing threads one
// block ahead, these 4-byte loads waited behind the bulk loads' queue: 538 us
// instead of the layer's 374 without sums (16384 tokens).
constexpr int kScaleSlots = 6;
constexpr int kMaxKBlocks = 64;          // d, F <= 8192
constexpr uint32_t kScaleBox = 132;
constexpr uint32_t kScaleSlotBytes = 640;

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
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

// Completion of a 32-column load, tied to its registers.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// acc += (v0, v1) * (f, f), two fp32 multiply-adds in one instruction.
__device__ __forceinline__ void fma2(float2& acc, uint32_t v0, uint32_t v1, uint64_t ff) {
  uint64_t a = *reinterpret_cast<uint64_t*>(&acc);
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}" : "+l"(a) : "r"(v0), "r"(v1), "l"(ff));
  acc = *reinterpret_cast<float2*>(&a);
}
__device__ __forceinline__ float2 mul2(uint32_t v0, uint32_t v1, uint64_t ff) {
  uint64_t a;
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tmul.rn.f32x2 %0, v, %3;\n\t}" : "=l"(a) : "r"(v0), "r"(v1), "l"(ff));
  return *reinterpret_cast<float2*>(&a);
}
__device__ __forceinline__ uint64_t twice(float f) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "r"(__float_as_uint(f)));
  return r;
}

// Instruction descriptor, kind::f8f6f4: D fp32, A and B E4M3, both K-major.
constexpr uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// SiLU(g) u: a few fp32 units off, far below the step of e4m3 (and more than the
// one rounding by which h (448 / amax) differs from the quotient by the scale).  g
// far below zero gives -0 (the exponential overflows, its reciprocal is 0).
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * rcp_fast(1.0f + exp2_fast(g * -kLog2e)) * u;
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// 64 bytes of each of the warp's 32 rows (lane l holds row l's) to dst + l *
// pitch, l < rows, by way of the warp's shared-memory buffer.
template <int kOutPitch>
__device__ __forceinline__ void store_rows(uint8_t* buf, const uint4 (&v)[4], uint8_t* dst, int64_t pitch, int rows) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + lane * kOutPitch + 16 * i) = v[i];
  __syncwarp();
  const int l0 = lane / 4, piece = (lane % 4) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int l = 8 * i + l0;
    const uint4 w = *reinterpret_cast<const uint4*>(buf + l * kOutPitch + piece);
    if (l < rows) *reinterpret_cast<uint4*>(dst + l * pitch + piece) = w;
  }
  __syncwarp();
}

// A 32 x 128 byte box in the swizzled layout of a TMA store (row l at 128 l,
// its 16-byte piece i at place i ^ (l % 8)): the first `rows` rows to dst.
__device__ __forceinline__ void store_box_rows(const uint8_t* box, uint8_t* dst, int64_t pitch, int rows) {
  const int lane = threadIdx.x & 31, piece = lane % 8;
  for (int l = lane / 8; l < rows; l += 4)
    *reinterpret_cast<uint4*>(dst + l * pitch + piece * 16) =
        *reinterpret_cast<const uint4*>(box + l * 128 + ((piece ^ (l & 7)) << 4));
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

// The tiles of a block, blockIdx.x, blockIdx.x + gridDim.x, ...: the group and
// feature block follow by steps, without a division or a search per tile
// (called by whole warps; 32 groups are looked at together).
struct F8Walk {
  const int32_t* mt;
  const int64_t* off;
  int G, n_tiles, dm, dn;
  int m, n, g;              // token block, feature block, group
  __device__ __forceinline__ F8Walk(const int32_t* mt_, const int64_t* off_, int G_, int n_tiles_)
      : mt(mt_), off(off_), G(G_), n_tiles(n_tiles_), g(0) {
    const int first = static_cast<int>(blockIdx.x), stride = static_cast<int>(gridDim.x);
    m = first / n_tiles;
    n = first - m * n_tiles;
    dm = stride / n_tiles;
    dn = stride - dm * n_tiles;
    seek();
  }
  __device__ __forceinline__ bool valid() const { return m < mt[G]; }
  __device__ __forceinline__ void seek() {          // g: the last group with mt[g] <= m
    while (true) {
      const int j = g + 1 + static_cast<int>(threadIdx.x & 31);
      const uint32_t le = __ballot_sync(0xffffffffu, j < G && mt[j] <= m);
      g += __popc(le);
      if (le != 0xffffffffu) break;
    }
  }
  __device__ __forceinline__ void step() {
    m += dm;
    n += dn;
    if (n >= n_tiles) {
      n -= n_tiles;
      ++m;
    }
    seek();
  }
  __device__ __forceinline__ int64_t row0() const { return off[g] + static_cast<int64_t>(m - mt[g]) * kTokRows; }
  __device__ __forceinline__ int rows() const {     // rows of the tile that exist
    const int64_t left = off[g + 1] - row0();
    return static_cast<int>(left < kTokRows ? left : kTokRows);
  }
};

template <bool kGateUp>
__global__ void __launch_bounds__(kF8Threads, 1)
    expert_fp8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_as, const __grid_constant__ CUtensorMap tm_ws,
                      const __grid_constant__ CUtensorMap tm_sc, const __grid_constant__ CUtensorMap tm_o,
                      const Fp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int32_t mt_s[kF8Groups + 1];
  __shared__ int64_t off_s[kF8Groups + 1];
  __shared__ int32_t warp_tot[kF8Threads / 32];
  __shared__ float amax_s[2][kTokRows];
  __shared__ int4 tile_s[2];                          // first row, rows that exist (0: no more tiles), feature block
  __shared__ float ws_s[2][2][kMaxKBlocks];           // its weight scales by k block, two blocks of weight rows
  using C = F8Cfg<kGateUp>;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  // ring, output rows (boxes on multiples of 1024 bytes), scale slots (of 128), barriers
  const uint32_t outs = ring + kF8Stage * C::kStages;
  const uint32_t slots = outs + kSumWarps * C::kOutBytes;
  static_assert(kScaleSlotBytes % 128 == 0 && kF8Stage % 1024 == 0 && C::kOutBytes % (kGateUp ? 16 : 1024) == 0 &&
                    (kSumWarps * C::kOutBytes) % 128 == 0, "alignment of TMA copies");
  const F8Bars bars{slots + kScaleSlotBytes * kScaleSlots};
  uint8_t* const holder_ptr = smem_raw + (bars.holder() - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.E + p.shared;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.done(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bars.free(b), kSumWarps);
      mbar_init(bars.tile(b), 1);
      mbar_init(bars.told(b), kSumWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(bars.holder()) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // Rows that no tile of the block has stay zero: what stood there would be multiplied all the same, at a power
  // that lowers the GPU's clock (64 tokens in 384 experts: 179 -> 172 us, 195 -> 187 under the power cap).
  for (int i = threadIdx.x; i < C::kStages * static_cast<int>(kABytes / 16); i += kF8Threads) {
    const uint32_t at = ring + kF8Stage * (i / (kABytes / 16)) + 16u * (i % (kABytes / 16));
    *reinterpret_cast<uint4*>(smem_raw + (at - raw)) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  pdl_wait();
  f8_tile_prefix(p, G, mt_s, off_s, warp_tot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(holder_ptr);

  if (warp < 4) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8RegsLow));
   if (warp == 0) {
    // TMA: the weights, the grouped rows (boxes of 32, only those that exist) and their scales
    // weights that several token blocks read stay in L2 (16384 tokens: 443 + 302 -> 430 + 274 us); others go first
    const uint64_t pol_w = p.NK > static_cast<int64_t>(kTokRows) * p.E ? policy_evict_last() : policy_evict_first();
    const uint64_t pol_a = policy_evict_last();
    int stage = 0, slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (F8Walk walk(mt_s, off_s, G, p.n_tiles); walk.valid() && ok; walk.step()) {
      const int g = walk.g, n = walk.n;
      const int64_t row0 = walk.row0();
      const bool sh = g == p.E;
      const CUtensorMap* tw = sh ? &tm_ws : &tm_w;
      const CUtensorMap* ta = kGateUp && sh ? &tm_as : &tm_a;
      const int a0 = static_cast<int>(kGateUp && sh ? row0 - p.NK : row0);
      // the gate rows of 128 units and their up rows, or 256 columns
      const int w0 = (sh ? 0 : g * p.w_rows) + n * (kGateUp ? 128 : 256);
      const int w1 = w0 + (kGateUp ? p.w_rows / 2 : 128);
      const int boxes = (walk.rows() + 31) / 32;
      const int s0 = static_cast<int>(row0 & ~static_cast<int64_t>(3));
      const uint32_t bytes = kBBytes + 4096u * boxes + kScaleBox * 4u;
      for (int kb = 0; kb < p.k_blocks && lane == 0; ++kb) {
        if (!mbar_wait(bars.done(stage), phase ^ 1u)) { ok = false; break; }
        const uint32_t a_dst = ring + kF8Stage * stage, b_dst = a_dst + kABytes, bar = bars.full(stage);
        mbar_arrive_expect_tx(bar, bytes);
        tma_load_2d(b_dst, tw, kb * kKBlock, w0, bar, pol_w);
        tma_load_2d(b_dst + kBBytes / 2, tw, kb * kKBlock, w1, bar, pol_w);
        for (int i = 0; i < boxes; ++i) tma_load_2d(a_dst + 4096u * i, ta, kb * kKBlock, a0 + 32 * i, bar, pol_a);
        tma_load_2d(slots + kScaleSlotBytes * slot, &tm_sc, s0, kb, bar, pol_a);
        slot = (slot + 1) % kScaleSlots;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
   } else if (warp <= 2 && lane == 0) {
      // MMAs: one thread per TMEM buffer, so that one's waits and commits run under the other's
      // multiplications (the queue behind a thread is too short for that).  The uses of a buffer stay in one
      // thread: its barrier is waited for by parity, one use ahead at most.
      constexpr uint32_t idesc = make_idesc_e4m3(kTokRows, kWRows);
      const int buf = warp - 1;
      const int64_t total = static_cast<int64_t>(mt_s[G]) * p.n_tiles;
      const int64_t first = blockIdx.x, stride = gridDim.x;
      const int64_t blocks = first < total ? ((total - 1 - first) / stride + 1) * p.k_blocks : 0;   // k blocks
      int stage = buf;
      uint32_t phase = 0, buf_phase = 0;
      for (int64_t q = buf; q < blocks; q += 2) {
        // free first: it says that the sums of block q - 2 are done, so that the stage's last use (q - 3 or before)
        // is, and full cannot be one phase behind the one that is waited for, which would look complete
        if (!mbar_wait(bars.free(buf), buf_phase ^ 1u) || !mbar_wait(bars.full(stage), phase)) break;
        const uint32_t a_addr = ring + kF8Stage * stage;
        const uint64_t a_desc = sw128_desc(a_addr), b_desc = sw128_desc(a_addr + kABytes);
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)           // 32 e4m3 along k = 32 bytes inside the swizzle row
          tc_mma_f8(tmem_base + 256u * buf, a_desc + 2u * ks, b_desc + 2u * ks, idesc, ks > 0 ? 1u : 0u);
        tc_commit(bars.done(stage));
        buf_phase ^= 1u;
        stage += 2;
        if (stage >= C::kStages) {
          stage -= C::kStages;
          phase ^= 1u;
        }
      }
   } else if (warp == 3) {
      // The tiles' places and weight scales for the sums, a tile ahead: worked out by the summing warps they cost
      // each tile a thousand cycles.
      const int wblocks = p.w_rows / 128;
      int t = 0;
      uint32_t phase = 0;
      F8Walk walk(mt_s, off_s, G, p.n_tiles);
      while (true) {
        const bool more = walk.valid();
        float w[kMaxKBlocks / 32][2];
        int4 place = make_int4(0, 0, 0, 0);
        if (more) {
          const float* w0 = (walk.g == p.E ? p.ws_scale : p.w_scale + static_cast<int64_t>(walk.g) * wblocks * p.k_blocks) +
                            static_cast<int64_t>(kGateUp ? walk.n : 2 * walk.n) * p.k_blocks;
          const float* w1 = w0 + static_cast<int64_t>(kGateUp ? wblocks / 2 : 1) * p.k_blocks;
#pragma unroll
          for (int i = 0; i < kMaxKBlocks / 32; ++i) {
            const int kb = lane + 32 * i;
            w[i][0] = kb < p.k_blocks ? __ldg(w0 + kb) : 0.0f;
            w[i][1] = kb < p.k_blocks ? __ldg(w1 + kb) : 0.0f;
          }
          place = make_int4(static_cast<int>(walk.row0()), walk.rows(), walk.n, 0);
        }
        if (!mbar_wait(bars.told(t), phase ^ 1u)) break;
#pragma unroll
        for (int i = 0; i < kMaxKBlocks / 32; ++i) {
          ws_s[t][0][lane + 32 * i] = w[i][0];
          ws_s[t][1][lane + 32 * i] = w[i][1];
        }
        if (lane == 0) tile_s[t] = place;
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.tile(t));
        if (!more) break;
        walk.step();
        if (++t == 2) {
          t = 0;
          phase ^= 1u;
        }
      }
   }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8RegsSum));
    // sums: thread = token row (TMEM lane quarter warp % 4), half of the columns.
    // Gate/up: half h holds the gates (columns 64 h) and the ups (128 + 64 h) of units 64 h .. 64 h + 63.
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t out_addr = outs + static_cast<uint32_t>((warp - 4) * C::kOutBytes);
    uint8_t* const out_s = smem_raw + (out_addr - raw);
    const uint32_t t_warp = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + (kGateUp ? 64u : 128u) * half;
    const float* const slots_s = reinterpret_cast<const float*>(smem_raw + (slots - raw));
    int stage = 0, buf = 0, slot = 0, t = 0;
    uint32_t phase = 0, tile_phase = 0;
    bool ok = true;
    while (true) {
      if (!mbar_wait(bars.tile(t), tile_phase)) break;
      const int4 place = tile_s[t];
      const int n = place.z, valid = place.y;
      if (valid == 0) break;
      const int64_t row0 = place.x;
      const bool live = r < valid, warp_live = quarter * 32 < valid;
      const int64_t row = row0 + r;
      const int srow = (place.x & 3) + r;
      const float* const w0 = ws_s[t][kGateUp ? 0 : half];
      float2 acc[4][16];
      // one k block; the first sets the sums (a choice inside one loop body costs both instructions)
      auto add = [&](int kb, auto first) -> bool {
        if (!mbar_wait(bars.done(stage), phase)) return false;
        tc_fence_after();
        auto release = [&]() {           // the buffer's columns of this warp are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.free(buf));
        };
        if (warp_live) {
          // the next 32 columns are on their way while these are added
          const uint32_t t0 = t_warp + 256u * buf;
          const float sa = slots_s[slot * (kScaleSlotBytes / 4) + srow];
          const uint64_t f0 = twice(sa * w0[kb]), f1 = kGateUp ? twice(sa * w0[kMaxKBlocks + kb]) : f0;
          uint32_t v[2][32];
          tmem_ld32(t0, v[0]);
          tmem_wait_ld32(v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c < 3) tmem_ld32(t0 + (kGateUp && c >= 1 ? 64u : 0u) + 32u * (c + 1), v[(c + 1) & 1]);
            const uint64_t f = c < 2 ? f0 : f1;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if constexpr (decltype(first)::value) acc[c][i] = mul2(v[c & 1][2 * i], v[c & 1][2 * i + 1], f);
              else fma2(acc[c][i], v[c & 1][2 * i], v[c & 1][2 * i + 1], f);
            }
            if (c < 3) tmem_wait_ld32(v[(c + 1) & 1]);
            if (c == 2) release();
          }
        } else {
          release();
        }
        slot = (slot + 1) % kScaleSlots;
        buf ^= 1;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      ok = add(0, std::true_type{});
      for (int kb = 1; kb < p.k_blocks && ok; ++kb) ok = add(kb, std::false_type{});
      if (!ok) break;
      if (lane == 0) mbar_arrive(bars.told(t));
      t ^= 1;
      tile_phase ^= t == 0 ? 1u : 0u;
      const int out_rows = valid - quarter * 32;       // rows of this warp that exist (may be <= 0)
      const int64_t wrow = row0 + quarter * 32;
      if constexpr (kGateUp) {
        float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            acc[c][i].x = silu_mul(acc[c][i].x, acc[c + 2][i].x);
            acc[c][i].y = silu_mul(acc[c][i].y, acc[c + 2][i].y);
            m[i & 3] = fmaxf(m[i & 3], fmaxf(fabsf(acc[c][i].x), fabsf(acc[c][i].y)));
          }
        float amax = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
        amax_s[half][r] = amax;
        asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");      // the two halves of these rows
        amax = fmaxf(fmaxf(amax, amax_s[half ^ 1][r]), kF8AmaxMin);
        asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");      // the two halves of these rows
        const uint64_t qq = twice(__fdiv_rn(kF8Max, amax));
        uint4 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 a[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 h = acc[j >> 1][(j & 1) * 8 + i];
            a[i] = mul2(__float_as_uint(h.x), __float_as_uint(h.y), qq);
          }
          o[j] = make_uint4(pack_e4m3(a[0].x, a[0].y, a[1].x, a[1].y),
                            pack_e4m3(a[2].x, a[2].y, a[3].x, a[3].y),
                            pack_e4m3(a[4].x, a[4].y, a[5].x, a[5].y),
                            pack_e4m3(a[6].x, a[6].y, a[7].x, a[7].y));
        }
        store_rows<C::kOutPitch>(out_s, o, static_cast<uint8_t*>(p.out) + wrow * p.ncols + n * 128 + half * 64, p.ncols, out_rows);
        if (live && half == 0) p.out_scale[n * p.ld + row] = __fdiv_rn(amax, kF8Max);
      } else {
        // the thread's 128 columns in fp16, scaled by the power of two that puts their largest in [2^14, 2^15)
        float m[4] = {kF8AmaxMin, kF8AmaxMin, kF8AmaxMin, kF8AmaxMin};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) m[i & 3] = fmaxf(m[i & 3], fmaxf(fabsf(acc[c][i].x), fabsf(acc[c][i].y)));
        const uint32_t top = __float_as_uint(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]))) & 0x7f800000u;
        const uint64_t qq = twice(__uint_as_float((268u << 23) - top));
        if (lane == 0) bulk_wait_read<0>();          // the buffer's last box has been read
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a0 = acc[c / 4][4 * (c % 4) + i];
            const float2 a = mul2(__float_as_uint(a0.x), __float_as_uint(a0.y), qq);
            const __half2 b = __floats2half2_rn(a.x, a.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(out_s + 4096 * (c / 8) + lane * 128 + (((c % 8) ^ (lane & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        const int col = n * 256 + half * 128;
        if (out_rows >= 32) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_o, col, static_cast<int>(wrow), out_addr);
            tma_store_2d(&tm_o, col + 64, static_cast<int>(wrow), out_addr + 4096u);
            bulk_commit();
          }
        } else if (out_rows > 0) {
          __syncwarp();
          uint8_t* dst = static_cast<uint8_t*>(p.out) + (wrow * p.ncols + col) * 2;
          store_box_rows(out_s, dst, 2 * p.ncols, out_rows);
          store_box_rows(out_s + 4096, dst + 128, 2 * p.ncols, out_rows);
        }
        if (live) p.out_scale[row * (p.ncols / 128) + 2 * n + half] = __uint_as_float(top - (14u << 23));
      }
    }
    if (!kGateUp && lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
}

// x8 rows by grouped row and their scales transposed, a block per 32 grouped
// rows: xp[p] = x8[perm[p] / K] for p < NK, and st[b][p] = xs[token of p][b] for
// p < NK + N (the shared expert's rows are the tokens in order, read in place).
// A bad entry of perm is reported and gives token 0.
constexpr int kGatherRows = 32;
__global__ void __launch_bounds__(256) gather_fp8_kernel(const uint4* __restrict__ x8, const float* __restrict__ xs,
                                                         const int32_t* __restrict__ perm, int64_t NK, int64_t rows,
                                                         int K, int vecs, int k_blocks, int64_t ld,
                                                         uint4* __restrict__ xp, float* __restrict__ st) {
  __shared__ int32_t tok[kGatherRows];
  __shared__ float sc[64][kGatherRows + 1];
  pdl_wait();
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kGatherRows;
  const int n = static_cast<int>(rows - p0 < kGatherRows ? rows - p0 : kGatherRows);
  if (threadIdx.x < n) {
    const int64_t q = p0 + threadIdx.x;
    int64_t t = q - NK;
    if (q < NK) {
      const int32_t j = perm[q];
      const bool bad = j < 0 || j >= NK;
      if (bad) raise_status(kStatusBadInput);
      t = bad ? 0 : j / K;
    }
    tok[threadIdx.x] = static_cast<int32_t>(t);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < kGatherRows / 8; ++i) {
    const int r = warp + 8 * i;
    if (r >= n || p0 + r >= NK) break;
    const uint4* src = x8 + static_cast<int64_t>(tok[r]) * vecs;
    uint4* dst = xp + (p0 + r) * vecs;
#pragma unroll 5
    for (int c = lane; c < vecs; c += 32) dst[c] = __ldg(src + c);
  }
  for (int r = warp; r < n; r += 8)
    for (int b = lane; b < k_blocks; b += 32) sc[b][r] = __ldg(xs + static_cast<int64_t>(tok[r]) * k_blocks + b);
  __syncthreads();
  for (int b = warp; b < k_blocks; b += 8)
    if (lane < n) st[b * ld + p0 + lane] = sc[b][lane];
}

// y[t] = o[NK + t] (shared) + sum_k gates[t,k] o[inv[t K + k]], fp32
// multiply-adds in the order shared, k ascending; a block per token, eight
// columns per thread, all KS = K + shared rows loaded before the first is added.
constexpr int kCombineThreads = 1024;    // d = 8192
template <int KS>
__global__ void __launch_bounds__(kCombineThreads) combine_fp8_kernel(const uint4* o, const float* os, const int32_t* inv,
                                                                      const float* gates, int64_t N, int K, int64_t NK,
                                                                      int vecs, uint4* y) {
  __shared__ int64_t slot[KS];
  __shared__ float gate[KS];
  const int shared = KS - K;
  pdl_wait();
  const int64_t t = blockIdx.x;
  if (threadIdx.x < KS) {
    const int k = static_cast<int>(threadIdx.x) - shared;
    int64_t q = NK + t;
    float g = 1.0f;
    if (k >= 0) {
      q = __ldg(inv + t * K + k);
      g = __ldg(gates + t * K + k);
      if (q < 0 || q >= NK) {
        raise_status(kStatusBadInput);
        q = 0;
      }
    }
    slot[threadIdx.x] = q;
    gate[threadIdx.x] = g;
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= vecs) return;
  uint4 v[KS];
  float s[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    v[k] = __ldg(o + slot[k] * vecs + c);
    s[k] = __ldg(os + slot[k] * (vecs / 16) + c / 16);
  }
  float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const float f = gate[k] * s[k];                // exact: s is a power of two
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      a[2 * i] = __fmaf_rn(f, h.x, a[2 * i]);
      a[2 * i + 1] = __fmaf_rn(f, h.y, a[2 * i + 1]);
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

struct CombineArgs {
  const uint4* o;
  const float* os;
  const int32_t* inv;
  const float* gates;
  int64_t N;
  int K, ks, vecs;
  uint4* y;
};
template <int KS>
cudaError_t launch_combine_fp8(const CombineArgs& a, cudaStream_t s) {
  if (a.ks == KS)
    return launch_pdl(combine_fp8_kernel<KS>, dim3(static_cast<unsigned>(a.N)), dim3((a.vecs + 31) / 32 * 32), 0, s,
                      dim3(0, 0, 0), a.o, a.os, a.inv, a.gates, a.N, a.K, a.N * a.K, a.vecs, a.y);
  if constexpr (KS < KOLIBRI_MAX_TOPK + 1) return launch_combine_fp8<KS + 1>(a, s);
  return cudaErrorInvalidValue;
}

template <bool kGateUp>
cudaError_t launch_fp8_gemm(const void* a, int64_t a_rows, const void* a_shared, int64_t as_rows, const void* w,
                            const void* w_shared, const float* scales, const Fp8Params& p, cudaStream_t s) {
  const uint64_t kdim = static_cast<uint64_t>(p.k_blocks) * kKBlock;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap tm_a, tm_w, tm_as, tm_ws, tm_sc, tm_o;
  if (!encode_2d(&tm_a, u8, 1, a, kdim, static_cast<uint64_t>(a_rows), kKBlock, 32) ||
      !encode_2d(&tm_as, u8, 1, a_shared, kdim, static_cast<uint64_t>(as_rows), kKBlock, 32) ||
      !encode_2d(&tm_w, u8, 1, w, kdim, static_cast<uint64_t>(p.E) * p.w_rows, kKBlock, 128) ||
      !encode_2d(&tm_ws, u8, 1, w_shared ? w_shared : w, kdim, static_cast<uint64_t>(p.w_rows), kKBlock, 128) ||
      !encode_2d(&tm_sc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, scales, static_cast<uint64_t>(p.ld),
                 static_cast<uint64_t>(p.k_blocks), kScaleBox, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      (!kGateUp && !encode_2d(&tm_o, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p.out, static_cast<uint64_t>(p.ncols),
                              static_cast<uint64_t>(p.NK + (p.shared ? p.N : 0)), 64, 32)))
    return cudaErrorInvalidValue;
  if (kGateUp) tm_o = tm_a;            // not used
  auto kern = expert_fp8_kernel<kGateUp>;
  using C = F8Cfg<kGateUp>;
  const size_t smem = 1024 + static_cast<size_t>(kF8Stage) * C::kStages + kScaleSlots * kScaleSlotBytes + kF8BarBytes +
                      kSumWarps * C::kOutBytes;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  // token blocks: at most one partial block per group that has rows
  const int64_t rows = p.NK + (p.shared ? p.N : 0);
  const int64_t partial = p.NK < p.E ? p.NK : p.E;
  const int64_t tiles = (rows / kTokRows + partial + p.shared) * p.n_tiles;
  const int64_t sms = device_sm_count();
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(kF8Threads), smem, s,
                    dim3(0, 0, 0), tm_a, tm_w, tm_as, tm_ws, tm_sc, tm_o, p);
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// h8 first: the hidden units in e4m3, then their scales, transposed.
struct Fp8Layout {
  int64_t rows, ld;         // grouped rows; ld: a multiple of 4, at least a scale box
  size_t off_h8, off_hs, off_x, off_xs, off_o, off_os, total;
};
Fp8Layout fp8_layout(int64_t N, int32_t d, int32_t F, int32_t K, bool shared) {
  Fp8Layout L{};
  L.rows = N * K + (shared ? N : 0);
  L.ld = (L.rows + 3) / 4 * 4;
  if (L.ld < static_cast<int64_t>(kScaleBox)) L.ld = kScaleBox;
  const size_t rows = static_cast<size_t>(L.rows), ld = static_cast<size_t>(L.ld);
  L.off_h8 = 0;
  L.off_hs = up256(rows * F);
  L.off_x = L.off_hs + up256(ld * (F / 128) * sizeof(float));
  L.off_xs = L.off_x + up256(static_cast<size_t>(N) * K * d);
  L.off_o = L.off_xs + up256(ld * (d / 128) * sizeof(float));
  L.off_os = L.off_o + up256(rows * d * sizeof(uint16_t));
  L.total = L.off_os + up256(rows * (d / 128) * sizeof(float));
  return L;
}

}  // namespace

bool expert_fp8_shape_supported(int32_t d, int32_t F, int32_t E) {
  return d >= 256 && d % 256 == 0 && d <= 8192 && F >= 128 && F % 128 == 0 && F <= 8192 && E >= 1 &&
         E <= KOLIBRI_MAX_EXPERTS && static_cast<int64_t>(E) * 2 * F < (1LL << 31) &&
         static_cast<int64_t>(E) * d < (1LL << 31);
}

size_t expert_fp8_ws_bytes(int64_t N, int32_t d, int32_t F, int32_t K, bool shared) {
  const Fp8Layout L = fp8_layout(N, d, F, K, shared);
  const size_t decode = static_cast<size_t>(L.rows) * F * sizeof(float);      // h in fp32
  return expert_fp8_decode_preferred(N, K, shared) && decode > L.total ? decode : L.total;
}

cudaError_t launch_expert_ffn_fp8(const ExpertFp8Args& a, cudaStream_t s) {
  const bool shared = a.ws_gate_up != nullptr;
  if (expert_fp8_decode_preferred(a.N, a.K, shared)) return launch_expert_ffn_fp8_decode(a, s);
  const Fp8Layout L = fp8_layout(a.N, a.d, a.F, a.K, shared);
  char* base = static_cast<char*>(a.ws);
  const int64_t NK = a.N * a.K;
  cudaError_t err = launch_pdl(
      gather_fp8_kernel, dim3(static_cast<unsigned>((L.rows + kGatherRows - 1) / kGatherRows)), dim3(256), 0, s,
      dim3(0, 0, 0), static_cast<const uint4*>(a.x8), a.x_scale, a.perm, NK, L.rows, a.K, a.d / 16, a.d / 128, L.ld,
      reinterpret_cast<uint4*>(base + L.off_x), reinterpret_cast<float*>(base + L.off_xs));
  if (err != cudaSuccess) return err;
  Fp8Params p{};
  p.offsets = a.offsets;
  p.N = a.N;
  p.NK = NK;
  p.ld = L.ld;
  p.E = a.E;
  p.shared = shared ? 1 : 0;
  p.w_scale = a.s_gate_up;
  p.ws_scale = a.ss_gate_up;
  p.out = base + L.off_h8;
  p.out_scale = reinterpret_cast<float*>(base + L.off_hs);
  p.k_blocks = a.d / 128;
  p.n_tiles = a.F / 128;
  p.ncols = a.F;
  p.w_rows = 2 * a.F;
  err = launch_fp8_gemm<true>(base + L.off_x, NK, a.x8, a.N, a.w_gate_up, a.ws_gate_up,
                              reinterpret_cast<const float*>(base + L.off_xs), p, s);
  if (err != cudaSuccess) return err;
  p.w_scale = a.s_down;
  p.ws_scale = a.ss_down;
  p.out = base + L.off_o;
  p.out_scale = reinterpret_cast<float*>(base + L.off_os);
  p.k_blocks = a.F / 128;
  p.n_tiles = a.d / 256;
  p.ncols = a.d;
  p.w_rows = a.d;
  err = launch_fp8_gemm<false>(base + L.off_h8, L.rows, base + L.off_h8, L.rows, a.w_down, a.ws_down,
                               reinterpret_cast<const float*>(base + L.off_hs), p, s);
  if (err != cudaSuccess) return err;
  const CombineArgs c{reinterpret_cast<const uint4*>(base + L.off_o), reinterpret_cast<const float*>(base + L.off_os),
                      a.inv, a.gates, a.N, a.K, a.K + (shared ? 1 : 0), a.d / 8, static_cast<uint4*>(a.y)};
  return launch_combine_fp8<1>(c, s);
}

KOLIBRI_DEFINE_STATUS_TAKE(status_take_expert_fp8)

}  // namespace kolibri
