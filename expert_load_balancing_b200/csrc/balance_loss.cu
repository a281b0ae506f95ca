// balance_loss.cu -- the auxiliary balance loss over the router's scores, the
// per-expert counts it weighs them with, and its gradient to the logits.
//
// The loss that "Kolibri Pre-Training from Scratch" 6.2 and 7 set Exact
// Quantile Balancing against.  Per sequence of T tokens (or once over a batch):
//
//   p_te = q_te / sum_j q_tj       q = exp(z) (softmax) or sigma(z) (the router's gate)
//   f_e  = E c_e / (K T)           c_e = slots of the sequence routed to e
//   P_e  = mean_t p_te,            L = lambda sum_e f_e P_e
//   dL/dz_te = lambda / T p_te (f_e - sum_j f_j p_tj) (1 - sigma(z_te) with sigmoid scores)
//
// The counts carry no gradient (they come from the selection).  As sum_j p_tj
// = 1, f enters as f - 1 throughout, which keeps the difference in the bracket
// exact to fp32 when the loads are nearly even: dot_t = sum_j (f_j - 1) p_tj,
// and at even loads L is lambda and the gradient 0 to the last bit.
//
// Measured (E = 384, 6 of them chosen, loss and gradient): 1,048,576 rows 564-572
// us, 0.87 of a copy's bandwidth for the 3.25 GB: counts 13, the pass 540-550, the
// finish 7.
//
// The gradient needs f, which comes from the ids alone, and not P: so with the
// gradient the counts are formed first (a read of the ids) and ONE pass over Z
// then forms P and dL/dZ.  Without it nothing in the pass needs f, and the pass
// counts too.  L = lambda (1 - r + sum_e (f_e - 1) P_e) comes from the sums of
// both, where r is the share of rows without p.  Bound by HBM: 4 E bytes of Z
// read and, with the gradient, 4 E bytes written per token.
//
// Sums over tokens: fp32 per warp over the rows of one block, then the blocks'
// shares in fp64 in a fixed order; counts are integers.  Nothing depends on
// the order in which blocks run.
//
// A block's chunk of rows may hold several sequences and a sequence may span
// several chunks.  The (chunk c, sequence s) pairs that meet form a staircase
// on which c + s never repeats, so the share of a pair is kept in row c + s of
// the workspace.
#include "launch.h"
#include "approx.cuh"
#include "common.cuh"
#include "pdl.cuh"

namespace kolibri {

namespace {

constexpr int kLossWarps = 8;
constexpr int kLossThreads = 32 * kLossWarps;
constexpr int kSmallWarps = 16;          // of the small form, whose eight blocks have an SM each
constexpr int kSmallThreads = 32 * kSmallWarps;
constexpr int kCountAhead = 8;           // ids in flight per thread of the counting pass
constexpr int kMaxE = KOLIBRI_MAX_EXPERTS;

constexpr int kSeqCache = 1024;

// Sequence boundaries: seq[0..S] (or null: one sequence of all rows), cut to
// [0, N] so that no index leaves the arrays whatever the caller wrote.
struct Seqs {
  const int64_t* seq;
  int64_t N;
  int S;
  // The same boundaries read from shared memory, if they fit: the search for a
  // block's first sequence is a chain of dependent loads.
  __device__ __forceinline__ Seqs cached(int64_t* buf) const {
    if (!seq || S >= kSeqCache) return *this;
    for (int s = threadIdx.x; s <= S; s += blockDim.x) buf[s] = seq[s];
    __syncthreads();
    return Seqs{buf, N, S};
  }
  __device__ __forceinline__ int64_t at(int s) const {
    if (!seq) return s == 0 ? 0 : N;
    const int64_t v = seq[s];
    return v < 0 ? 0 : (v > N ? N : v);
  }
  // the last s < S with at(s) <= row, or 0
  __device__ __forceinline__ int find(int64_t row) const {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (at(mid) <= row) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

// Offsets that decrease or leave [0, N] are reported (the blocks share them).
__device__ __forceinline__ void check_seqs(const Seqs& q) {
  if (q.seq)
    for (int64_t s = blockIdx.x * kLossThreads + threadIdx.x; s <= q.S; s += static_cast<int64_t>(gridDim.x) * kLossThreads) {
      const int64_t v = q.seq[s];
      if (v < 0 || v > q.N || (s > 0 && q.seq[s - 1] > v)) raise_status(kStatusBadInput);
    }
}

// hist[e] += the slots of the rows [lo, hi) that are routed to e.
template <int kThreads>
__device__ __forceinline__ void count_rows(const int32_t* ids, int64_t lo, int64_t hi, int E, int K, int32_t* hist) {
  const int64_t j1 = hi * K;
  for (int64_t j = lo * K + threadIdx.x; j < j1; j += kCountAhead * kThreads) {
    int32_t e[kCountAhead];
#pragma unroll
    for (int i = 0; i < kCountAhead; ++i)
      if (j + i * kThreads < j1) e[i] = __ldcs(ids + j + i * kThreads);
#pragma unroll
    for (int i = 0; i < kCountAhead; ++i)
      if (j + i * kThreads < j1) {
        if (e[i] >= 0 && e[i] < E) atomicAdd(&hist[e[i]], 1);
        else raise_status(kStatusBadInput);
      }
  }
}

// counts += hist, hist = 0.
__device__ __forceinline__ void flush_counts(int32_t* hist, int E, int32_t* counts) {
  for (int e = threadIdx.x; e < E; e += kLossThreads) {
    const int32_t c = hist[e];
    if (c) {
      atomicAdd(&counts[e], c);
      hist[e] = 0;
    }
  }
}

// counts [S][E] += the slots of this block's rows.  counts is zero on entry.
__global__ void __launch_bounds__(kLossThreads) seq_count_kernel(const int32_t* ids, Seqs given, int E, int K,
                                                                 int64_t chunk, int32_t* counts) {
  __shared__ int32_t hist[kMaxE];
  __shared__ int64_t seq_s[kSeqCache];
  const Seqs q = given.cached(seq_s);
  const int64_t r0 = blockIdx.x * chunk;
  const int64_t r1 = r0 + chunk < q.N ? r0 + chunk : q.N;
  for (int e = threadIdx.x; e < E; e += kLossThreads) hist[e] = 0;
  check_seqs(q);
  __syncthreads();
  for (int s = q.find(r0); s < q.S; ++s) {
    const int64_t b = q.at(s), e_ = q.at(s + 1);
    if (b >= r1) break;
    const int64_t lo = b > r0 ? b : r0, hi = e_ < r1 ? e_ : r1;
    if (lo >= hi) continue;
    count_rows<kLossThreads>(ids, lo, hi, E, K, hist);
    __syncthreads();
    flush_counts(hist, E, counts + static_cast<int64_t>(s) * E);
    __syncthreads();
  }
}

struct LossParams {
  const float* z;
  const int32_t* ids;       // [N, K]: counted in the pass without the gradient
  int32_t* counts;          // [S, E]
  const float* grad_loss;   // [S] or null (ones)
  float* gz;                // [N, E]
  float* part;              // [chunks + S][E]: sums of p
  double* none;             // [chunks + S]: rows without p
  Seqs q;
  int64_t chunk;
  int E, K;
  int accumulate;
  double lambda;
};

// The product with log2 e adds 2^-24 |z - c| to exp2_fast's error; all far below
// the 2^-24 sqrt(T) of the sums the scores enter.  (c is subtracted first:
// folded into one multiply-add it would cost 2^-24 of |z| for logits far from
// zero.)

// L lanes per row (8, 16 or 32): lane l of them holds the float4s l, l + L, ...
// (V of them) of the row's E logits.  Narrow rows share a warp, so that a row's
// reductions cost it a share of the shuffles only: a warp per row of 128 logits
// spent 149 instructions a row, most of them there (E = 128, 65,536 rows in 61
// sequences, loss and gradient apart: 46 us).
//
// Sigmoid scores are formed as q = 1 / (e^c + e^(c - z)) = e^-c sigma(z) with c
// = min(max_j z_j, 0): the common factor keeps rows whose logits are all far
// below zero from vanishing.  1 - sigma(z) = q e^(c - z) where sigma > 1/2 and
// 1 - q e^c elsewhere, both free of cancellation.  A row without a finite
// logit gives p = 0 and gradient 0.
//
// Blocks per SM: the warps that wait for loads count (E = 384, 1M rows, loss
// and gradient: 575 us at four blocks, 640 at two, 765 at the three of an
// unbounded register count).  With four float4s a lane the sums and logits need
// more than the 64 registers of four blocks, and two without spills beat three
// with at every such width (262,144 rows, sigmoid scores, loss and gradient at
// once, in a graph: E = 128 64 us at two and 91 at three, 256 105 and 155, 512 188
// and 308; E = 128, 65,536 rows in 61 sequences, loss and then gradient: 34 and 38).
template <int V>
struct LossBlocks {
  static constexpr int kPerSm = V <= 3 ? 4 : 2;
};

// Rows [lo, hi) of sequence s, which is rows [b, e_), with its counts: writes
// their gradient, and leaves the warps' shares of P in psum and of sum dot (kDots)
// or of the number of rows without p in dsum (all threads of the block; ends with
// a barrier if kProb).
template <int L, int V, bool kSoftmax, bool kProb, bool kGrad, bool kDots>
__device__ __forceinline__ void loss_rows(const LossParams& p, const int32_t* counts, int s, int64_t b, int64_t e_,
                                          int64_t lo, int64_t hi, float* psum, double* dsum) {
  constexpr int kRows = 32 / L;          // rows of a warp at once
  constexpr int kWarps = kDots ? kSmallWarps : kLossWarps;
  // The next rows are on their way while these are worked on, where the registers are there for it (65,536 rows of
  // 128, two blocks per SM: the gradient's pass 13.9 -> 12.4 us, the other 17.1 -> 16.3).
  constexpr bool kAhead = V == 4;
  const int lane = threadIdx.x & (L - 1), group = (threadIdx.x & 31) / L, warp = threadIdx.x >> 5;
  const int E4 = p.E >> 2;
  // f - 1 = (E c - K T) / (K T), the numerator an integer: exact where loads are even
  const int64_t slots = (e_ - b) * p.K;
  const float per_slot = __fdiv_rn(1.0f, static_cast<float>(slots));
  float fr[4 * V], acc[4 * V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c4 = lane + L * j;
    int4 c = make_int4(0, 0, 0, 0);
    if ((kGrad || kDots) && c4 < E4) c = reinterpret_cast<const int4*>(counts)[c4];
    fr[4 * j + 0] = static_cast<float>(static_cast<int64_t>(c.x) * p.E - slots) * per_slot;
    fr[4 * j + 1] = static_cast<float>(static_cast<int64_t>(c.y) * p.E - slots) * per_slot;
    fr[4 * j + 2] = static_cast<float>(static_cast<int64_t>(c.z) * p.E - slots) * per_slot;
    fr[4 * j + 3] = static_cast<float>(static_cast<int64_t>(c.w) * p.E - slots) * per_slot;
  }
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) acc[i] = 0.0f;
  float gscale = 0.0f;
  if constexpr (kGrad)
    gscale = __fdiv_rn(static_cast<float>(p.lambda) * (p.grad_loss ? p.grad_loss[s] : 1.0f), static_cast<float>(e_ - b));
  double dot_sum = 0.0;
  float4 next[V];
  auto fetch = [&](int64_t row) {
    const float4* zr = reinterpret_cast<const float4*>(p.z) + row * E4;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c4 = lane + L * j;
      next[j] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (c4 < E4 && row < hi) next[j] = __ldcs(zr + c4);
    }
  };
  if (kAhead) fetch(lo + warp * kRows + group);
  for (int64_t base = lo + warp * kRows; base < hi; base += kRows * kWarps) {
    const int64_t row = base + group;
    const bool there = row < hi;
    if (!kAhead) fetch(row);
    float z[4 * V], u[4 * V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      z[4 * j] = next[j].x; z[4 * j + 1] = next[j].y; z[4 * j + 2] = next[j].z; z[4 * j + 3] = next[j].w;
    }
    if (kAhead) fetch(row + kRows * kWarps);
    float m = z[0];
#pragma unroll
    for (int i = 1; i < 4 * V; ++i) m = fmaxf(m, z[i]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool low = m == -INFINITY;
    float sum = 0.0f, dot = 0.0f, ec = 1.0f;
    if constexpr (kSoftmax) {
      const float c = low ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) z[i] = exp2_fast((z[i] - c) * kLog2e);
    } else {
      const float c = low ? 0.0f : fminf(m, 0.0f);
      ec = exp2_fast(c * kLog2e);
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) {
        u[i] = exp2_fast((c - z[i]) * kLog2e);
        z[i] = rcp_fast(ec + u[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) {
      sum += z[i];
      dot = fmaf(fr[i], z[i], dot);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    // A row of -infinity throughout, as a row behind the last one is.  The score at the maximum is 1/2 at least, so no
    // other sum is 0.  The maximum does not tell: it passes over NaN, and a row of NaN has to show in P and L.
    const bool none = sum == 0.0f;
    const float inv = none ? 0.0f : rcp_fast(sum);
    dot = __fmul_rn(dot, inv);          // uncontracted: the same bits in every form of the pass
    if constexpr (kProb) {
      if constexpr (kDots) dot_sum += !there ? 0.0f : none ? -1.0f : dot;       // a row without p adds nothing to L
      else dot_sum += there && none ? 1.0f : 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) acc[i] = fmaf(z[i], inv, acc[i]);
    }
    if constexpr (kGrad) {
      const float k = gscale * inv;
      float4* gr = reinterpret_cast<float4*>(p.gz) + row * E4;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c4 = lane + L * j;
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = 4 * j + i;
          o[i] = k * z[x] * (fr[x] - dot);
          if constexpr (!kSoftmax) o[i] *= u[x] < ec ? z[x] * u[x] : fmaf(-z[x], ec, 1.0f);
        }
        if (c4 < E4 && there) {
          if (p.accumulate) {
            const float4 old = gr[c4];
            o[0] += old.x; o[1] += old.y; o[2] += old.z; o[3] += old.w;
          }
          __stcs(gr + c4, make_float4(o[0], o[1], o[2], o[3]));
        }
      }
    }
  }
  if constexpr (kProb) {
    // the warp's rows at once, in a fixed order
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      dot_sum += __shfl_xor_sync(0xffffffffu, dot_sum, o);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c4 = lane + L * j;
      if (c4 < E4 && group == 0)
        reinterpret_cast<float4*>(psum + warp * kMaxE)[c4] =
            make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
    }
    if (lane == 0 && group == 0) dsum[warp] = dot_sum;
    __syncthreads();
  }
}

// kProb && !kGrad: the pass counts too; counts is zero on entry.
template <int L, int V, bool kSoftmax, bool kProb, bool kGrad>
__global__ void __launch_bounds__(kLossThreads, LossBlocks<V>::kPerSm) balance_loss_kernel(const LossParams p) {
  constexpr bool kCount = kProb && !kGrad;
  __shared__ float psum[kProb ? kLossWarps * kMaxE : 1];
  __shared__ int32_t hist[kCount ? kMaxE : 1];
  __shared__ double dsum[kLossWarps];
  const int E4 = p.E >> 2;
  __shared__ int64_t seq_s[kSeqCache];
  const int64_t r0 = blockIdx.x * p.chunk;
  const int64_t r1 = r0 + p.chunk < p.q.N ? r0 + p.chunk : p.q.N;
  pdl_wait();          // the counts
  const Seqs q = p.q.cached(seq_s);
  if constexpr (kCount || !kProb) check_seqs(q);       // the other form's counting pass has checked them
  if constexpr (kCount) {
    for (int e = threadIdx.x; e < p.E; e += kLossThreads) hist[e] = 0;
    __syncthreads();
  }
  if constexpr (kGrad) {
    // rows of the chunk before the first and behind the last sequence have no gradient
    if (!p.accumulate) {
      const int64_t first = q.at(0), last = q.at(q.S);
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      float4* g4 = reinterpret_cast<float4*>(p.gz);
      const int64_t a1 = first < r1 ? first : r1, b0 = last > r0 ? last : r0;
      for (int64_t i = r0 * E4 + threadIdx.x; i < a1 * E4; i += kLossThreads) g4[i] = zero;
      for (int64_t i = b0 * E4 + threadIdx.x; i < r1 * E4; i += kLossThreads) g4[i] = zero;
    }
  }
  for (int s = q.find(r0); s < q.S; ++s) {
    const int64_t b = q.at(s), e_ = q.at(s + 1);
    if (b >= r1) break;
    const int64_t lo = b > r0 ? b : r0, hi = e_ < r1 ? e_ : r1;
    if (lo >= hi) continue;
    int32_t* const counts = p.counts + static_cast<int64_t>(s) * p.E;
    if constexpr (kCount) count_rows<kLossThreads>(p.ids, lo, hi, p.E, p.K, hist);
    loss_rows<L, V, kSoftmax, kProb, kGrad, false>(p, counts, s, b, e_, lo, hi, psum, dsum);
    if constexpr (kCount) flush_counts(hist, p.E, counts);
    if constexpr (kProb) {
      const int64_t slot = blockIdx.x + s;
      for (int e = threadIdx.x; e < p.E; e += kLossThreads) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kLossWarps; ++w) t += psum[w * kMaxE + e];
        p.part[slot * p.E + e] = t;
      }
      if (threadIdx.x == 0) {
        double t = 0.0;
#pragma unroll
        for (int w = 0; w < kLossWarps; ++w) t += dsum[w];
        p.none[slot] = t;
      }
      __syncthreads();
    }
  }
}

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ double remote_f64(const void* p, uint32_t rank) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// prob[s][e] and loss[s] from the blocks' shares and the counts: a cluster per
// sequence, a block of it per 64 experts, 16 shares at a time, fp64, fixed order.
constexpr int kFinishRows = 16;
constexpr int kFinishCols = 64;
static_assert(kMaxE / kFinishCols <= 8, "a cluster of at most eight blocks");
__global__ void __launch_bounds__(32 * kFinishRows) balance_finish_kernel(const LossParams p, float* prob, float* loss) {
  __shared__ double buf[kFinishRows][kFinishCols];
  __shared__ double dot_s;
  pdl_wait();
  const int tiles = (p.E + kFinishCols - 1) / kFinishCols;
  const int s = blockIdx.x / tiles, tile = blockIdx.x - s * tiles;       // tile: the rank in the cluster
  const int e = tile * kFinishCols + 2 * threadIdx.x;                    // and e + 1: E is a multiple of 4
  const int64_t b = p.q.at(s), en = p.q.at(s + 1);
  const int64_t n = en > b ? en - b : 0;
  const int64_t c0 = n ? b / p.chunk : 0, c1 = n ? (en - 1) / p.chunk + 1 : 0;   // chunks that hold rows of s
  double t0 = 0.0, t1 = 0.0;
  if (e < p.E)
#pragma unroll 4
    for (int64_t c = c0 + threadIdx.y; c < c1; c += kFinishRows) {
      const float2 v = *reinterpret_cast<const float2*>(p.part + (c + s) * p.E + e);
      t0 += v.x;
      t1 += v.y;
    }
  buf[threadIdx.y][2 * threadIdx.x] = t0;
  buf[threadIdx.y][2 * threadIdx.x + 1] = t1;
  double none = 0.0;                     // of the last warp: its chain runs beside the first one's
  if (threadIdx.y == kFinishRows - 1 && tile == 0) {
    for (int64_t c = c0 + threadIdx.x; c < c1; c += 32) none += p.none[c + s];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) none += __shfl_xor_sync(0xffffffffu, none, o);
  }
  __syncthreads();
  if (threadIdx.y == 0) {
    double dot = 0.0;
    if (e < p.E) {
      t0 = t1 = 0.0;
#pragma unroll
      for (int r = 0; r < kFinishRows; ++r) {
        t0 += buf[r][2 * threadIdx.x];
        t1 += buf[r][2 * threadIdx.x + 1];
      }
      const double mean = n ? 1.0 / static_cast<double>(n) : 0.0;
      t0 *= mean;
      t1 *= mean;
      *reinterpret_cast<float2*>(prob + static_cast<int64_t>(s) * p.E + e) =
          make_float2(static_cast<float>(t0), static_cast<float>(t1));
      const int2 c = *reinterpret_cast<const int2*>(p.counts + static_cast<int64_t>(s) * p.E + e);
      const int64_t slots = n * p.K;
      dot = static_cast<double>(static_cast<int64_t>(c.x) * p.E - slots) * t0 +
            static_cast<double>(static_cast<int64_t>(c.y) * p.E - slots) * t1;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (threadIdx.x == 0) dot_s = dot;
  }
  cluster_barrier();
  if (tile == 0 && threadIdx.y == kFinishRows - 1 && threadIdx.x == 0) {
    double dot = 0.0;
    for (int r = 0; r < tiles; ++r) dot += remote_f64(&dot_s, r);
    const double rows = static_cast<double>(n);
    loss[s] = n ? static_cast<float>(p.lambda * (1.0 - none / rows + dot / (rows * p.K))) : 0.0f;
  }
  cluster_barrier();                     // no block leaves while another reads its shared memory
}

// A small batch of one sequence: one launch, a cluster of eight blocks that
// hold the counts and the shares of P in shared memory and read one another's.
// The launches of the other form cost 12.3 us whatever the size; 256 rows of 384
// take 7.3 here (9.0 with eight warps; 13.4 the other way), 64 rows 5.4 (in a graph
// of fifty calls, each on inputs of its own).  Eight SMs cannot carry more: 680 rows
// of 384 14.5 (14.8 the other way), 1024 18.9 (14.4); 512 rows of 512 12.4 (15.7),
// 1024 of 256 11.8 (15.3).
constexpr int kClusterBlocks = 8;
constexpr int64_t kSmallRows = 1024;
constexpr int64_t kSmallLogits = 1 << 18;
// Up to this many slots each block counts all ids: one round of loads in place of
// a barrier of the cluster and a round of remote ones (64 rows of 384, K = 6, eight
// warps: 5.1 us, 6.0 with the barrier; 680 rows: 15.6 and 15.8).
constexpr int64_t kAloneSlots = 4096;
bool small_batch(int64_t N, int32_t E, int32_t S) { return S == 1 && N <= kSmallRows && N * E <= kSmallLogits; }

template <int L, int V, bool kSoftmax, bool kGrad>
__global__ void __launch_bounds__(kSmallThreads) balance_small_kernel(const LossParams p, const int32_t* ids,
                                                                     int32_t* counts_out, float* prob, float* loss) {
  __shared__ float psum[kSmallWarps * kMaxE];
  __shared__ double dsum[kSmallWarps];
  __shared__ int32_t hist[kMaxE];
  __shared__ __align__(16) int32_t counts[kMaxE];
  __shared__ float share[kMaxE];
  __shared__ double dots;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  for (int e = threadIdx.x; e < p.E; e += kSmallThreads) hist[e] = 0;
  pdl_wait();
  const Seqs q = p.q;
  if (rank == 0 && threadIdx.x == 0 && q.seq && (q.seq[0] < 0 || q.seq[0] > q.seq[1] || q.seq[1] > q.N))
    raise_status(kStatusBadInput);
  const int64_t b = q.at(0), end = q.at(1), e_ = end > b ? end : b;
  const int64_t r0 = rank * p.chunk, r1 = r0 + p.chunk < q.N ? r0 + p.chunk : q.N;
  const int64_t lo = b > r0 ? b : r0, hi = e_ < r1 ? e_ : r1;
  __syncthreads();
  const bool alone = (e_ - b) * p.K <= kAloneSlots;
  if (alone) {
    count_rows<kSmallThreads>(ids, b, e_, p.E, p.K, hist);
    __syncthreads();
  } else {
    count_rows<kSmallThreads>(ids, lo, hi, p.E, p.K, hist);
    cluster_barrier();
  }
  for (int e = threadIdx.x; e < p.E; e += kSmallThreads) {
    int32_t c = 0;
    if (alone) {
      c = hist[e];
    } else {
#pragma unroll
      for (uint32_t r = 0; r < kClusterBlocks; ++r) c += static_cast<int32_t>(remote_u32(hist + e, r));
    }
    counts[e] = c;
    if (rank == 0) counts_out[e] = c;
  }
  __syncthreads();
  if constexpr (kGrad) {
    if (!p.accumulate)
      for (int64_t i = r0 * p.E + threadIdx.x; i < r1 * p.E; i += kSmallThreads)
        if (i < b * p.E || i >= e_ * p.E) p.gz[i] = 0.0f;
  }
  if (lo < hi) {
    loss_rows<L, V, kSoftmax, true, kGrad, true>(p, counts, 0, b, e_, lo, hi, psum, dsum);
  } else {
    if (threadIdx.x < kSmallWarps) dsum[threadIdx.x] = 0.0;
    for (int i = threadIdx.x; i < kSmallWarps * kMaxE; i += kSmallThreads) psum[i] = 0.0f;
    __syncthreads();
  }
  for (int e = threadIdx.x; e < p.E; e += kSmallThreads) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) t += psum[w * kMaxE + e];
    share[e] = t;
  }
  if (threadIdx.x == 0) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) t += dsum[w];
    dots = t;
  }
  cluster_barrier();
  const int64_t n = e_ - b;
  for (int e = rank * kSmallThreads + threadIdx.x; e < p.E; e += kClusterBlocks * kSmallThreads) {
    double t = 0.0;
#pragma unroll
    for (uint32_t r = 0; r < kClusterBlocks; ++r) t += __uint_as_float(remote_u32(share + e, r));
    prob[e] = n ? static_cast<float>(t / static_cast<double>(n)) : 0.0f;
  }
  if (rank == kClusterBlocks - 1 && threadIdx.x == 0) {
    double t = 0.0;
#pragma unroll
    for (uint32_t r = 0; r < kClusterBlocks; ++r) t += remote_f64(&dots, r);
    loss[0] = n ? static_cast<float>(p.lambda * (1.0 + t / static_cast<double>(n))) : 0.0f;
  }
  cluster_barrier();                     // no block leaves while another reads its shared memory
}

struct LossPlan {
  int64_t chunk, chunks;
};
// One wave of blocks: a second one, of a few blocks, cost 65,536 rows of 128
// half their time again.
LossPlan loss_plan(int64_t N, int32_t E) {
  const bool wide = (E > 64 && E <= 128) || (E > 192 && E <= 256) || E > 384;      // four float4s per lane
  const int64_t most = static_cast<int64_t>(device_sm_count()) * (wide ? LossBlocks<4>::kPerSm : LossBlocks<3>::kPerSm);
  LossPlan lp;
  lp.chunk = (N + most - 1) / most;
  lp.chunk = (lp.chunk + kLossWarps - 1) / kLossWarps * kLossWarps;
  lp.chunks = (N + lp.chunk - 1) / lp.chunk;
  return lp;
}

template <bool kProb, bool kGrad>
struct LossPass {
  int64_t chunks;           // without the counting pass in front of it an ordinary launch, behind a memset
  template <int L, int V>
  cudaError_t run(const LossParams& p, int score, cudaStream_t s) const {
    auto kern = score == KOLIBRI_SCORE_SOFTMAX ? balance_loss_kernel<L, V, true, kProb, kGrad>
                                               : balance_loss_kernel<L, V, false, kProb, kGrad>;
    if constexpr (kGrad) {
      return launch_pdl(kern, dim3(static_cast<unsigned>(chunks)), dim3(kLossThreads), 0, s, dim3(0, 0, 0), p);
    } else {
      kern<<<static_cast<unsigned>(chunks), kLossThreads, 0, s>>>(p);
      return cudaGetLastError();
    }
  }
};

struct SmallPass {
  const int32_t* ids;
  int32_t* counts;
  float* prob;
  float* loss;
  template <int L, int V, bool kSoftmax>
  cudaError_t launch(const LossParams& p, cudaStream_t s) const {
    auto kern = p.gz ? balance_small_kernel<L, V, kSoftmax, true> : balance_small_kernel<L, V, kSoftmax, false>;
    return launch_pdl(kern, dim3(kClusterBlocks), dim3(kSmallThreads), 0, s, dim3(kClusterBlocks, 1, 1), p, ids, counts,
                      prob, loss);
  }
  template <int L, int V>
  cudaError_t run(const LossParams& p, int score, cudaStream_t s) const {
    return score == KOLIBRI_SCORE_SOFTMAX ? launch<L, V, true>(p, s) : launch<L, V, false>(p, s);
  }
};

// The fewest lanes whose four float4s hold a row.
template <typename Pass>
cudaError_t launch_by_width(const Pass& pass, const LossParams& p, int score, cudaStream_t s) {
  if (p.E <= 64) return pass.template run<8, 2>(p, score, s);
  if (p.E <= 128) return pass.template run<8, 4>(p, score, s);
  if (p.E <= 192) return pass.template run<16, 3>(p, score, s);
  if (p.E <= 256) return pass.template run<16, 4>(p, score, s);
  if (p.E <= 384) return pass.template run<32, 3>(p, score, s);
  return pass.template run<32, 4>(p, score, s);
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t balance_loss_ws_bytes(int64_t N, int32_t E, int32_t S) {
  if (small_batch(N, E, S)) return 0;
  const size_t rows = static_cast<size_t>(loss_plan(N, E).chunks) + S;
  return round256(rows * E * sizeof(float)) + rows * sizeof(double);
}

cudaError_t launch_balance_loss(const float* z, const int32_t* ids, const int64_t* seq, int64_t N, int32_t E,
                                int32_t K, int32_t S, int score, double lambda, const float* grad_loss,
                                int accumulate, float* loss, int32_t* counts, float* prob, float* gz, void* ws,
                                cudaStream_t s) {
  const LossPlan lp = loss_plan(N, E);
  LossParams p{};
  p.z = z;
  p.ids = ids;
  p.counts = counts;
  p.grad_loss = grad_loss;
  p.gz = gz;
  p.part = static_cast<float*>(ws);
  p.none = reinterpret_cast<double*>(static_cast<char*>(ws) +
                                     round256((static_cast<size_t>(lp.chunks) + S) * E * sizeof(float)));
  p.q = Seqs{seq, N, S};
  p.chunk = lp.chunk;
  p.E = E;
  p.K = K;
  p.accumulate = accumulate;
  p.lambda = lambda;
  if (small_batch(N, E, S)) {
    p.chunk = (N + kClusterBlocks - 1) / kClusterBlocks;
    return launch_by_width(SmallPass{ids, counts, prob, loss}, p, score, s);
  }
  cudaError_t err = cudaMemsetAsync(counts, 0, sizeof(int32_t) * static_cast<size_t>(S) * E, s);
  if (err != cudaSuccess) return err;
  if (gz) {
    seq_count_kernel<<<static_cast<unsigned>(lp.chunks), kLossThreads, 0, s>>>(ids, p.q, E, K, lp.chunk, counts);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  err = gz ? launch_by_width(LossPass<true, true>{lp.chunks}, p, score, s)
           : launch_by_width(LossPass<true, false>{lp.chunks}, p, score, s);
  if (err != cudaSuccess) return err;
  const unsigned tiles = static_cast<unsigned>((E + kFinishCols - 1) / kFinishCols);
  return launch_pdl(balance_finish_kernel, dim3(tiles * static_cast<unsigned>(S)), dim3(32, kFinishRows), 0, s,
                    dim3(tiles, 1, 1), p, prob, loss);
}

cudaError_t launch_balance_loss_grad(const float* z, const int32_t* counts, const int64_t* seq, int64_t N,
                                     int32_t E, int32_t K, int32_t S, int score, double lambda,
                                     const float* grad_loss, int accumulate, float* gz, cudaStream_t s) {
  const LossPlan lp = loss_plan(N, E);
  LossParams p{};
  p.z = z;
  p.counts = const_cast<int32_t*>(counts);       // read only
  p.grad_loss = grad_loss;
  p.gz = gz;
  p.q = Seqs{seq, N, S};
  p.chunk = lp.chunk;
  p.E = E;
  p.K = K;
  p.accumulate = accumulate;
  p.lambda = lambda;
  return launch_by_width(LossPass<false, true>{lp.chunks}, p, score, s);
}

KOLIBRI_DEFINE_STATUS_TAKE(status_take_balance_loss)

}  // namespace kolibri
