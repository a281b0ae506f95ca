// norm.cu -- the norm in front of the router: root-mean-square norm of the
// residual stream with the residual's addition, a bf16 output for the router
// and an 8-bit output with scales for the experts, and its gradient.
//
// "Kolibri 1 im Detail", routing and FP8 sections: the router takes bf16
// tokens [N, 2560]; the experts' activations are E4M3 with one fp32 scale per
// 1 x 128 group.
//
//   h = x + res                       fp32; res_out = h rounded once to res's type
//   r = rsqrt(mean(h^2) + eps)        fp32, from the unrounded h
//   y = h r g                         fp32; rounded once to bf16
//   s = max(amax_group |y|, 1e-30) / 448,  y8 = e4m3(y / s)   from the fp32 y, each a rounded quotient
//
// Bound by HBM: each input is read once and each output written once, the
// row stays in registers between the sum of squares and the outputs.  Measured:
// 16,384 rows of 2560 (bf16 in, residual, bf16 and 8-bit out, 379 MB) 62 us, 0.94
// of a copy's bandwidth; 65,536 rows of 2048 (fp32 residual, 1.61 GB) 236 us,
// 1.04; the gradient of 16,384 rows of 2560 (335 MB) 58 us, 0.89, and 4 for the
// weight's sum; a row of one token 4.2 us in a graph of its own, the latency of a
// launch, one round of reads (none waits for another) and a block's sum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <type_traits>

#include "launch.h"
#include "approx.cuh"
#include "common.cuh"
#include "pdl.cuh"

namespace kolibri {

namespace {

constexpr int kVec = 8;                  // elements per thread and step: 16 bytes of bf16
constexpr int kGroupVecs = 128 / kVec;   // threads of one 8-bit scale group
constexpr int kMaxNormThreads = 1024;   // d = 16384 at two vecs per thread
constexpr int kMaxNormWarps = kMaxNormThreads / 32;
constexpr float kAmaxMin = 1e-30f;       // keeps the scale and its reciprocal normal numbers

struct Vec8 {
  float v[kVec];
};

// Eight elements as they lie in memory: 16 bytes of bf16, 32 of fp32.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const void* p, int64_t vec) {
  Raw8<T> r;
  const uint4* q = reinterpret_cast<const uint4*>(p) + vec * (sizeof(T) / 2);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = q[i];
  return r;
}

template <typename T>
__device__ __forceinline__ Vec8 widen(const Raw8<T>& r) {
  Vec8 o;
  if constexpr (sizeof(T) == 2) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[2 * i] = __uint_as_float(w[i] << 16);
      o.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __uint_as_float(w[i]);
  }
  return o;
}

template <typename T>
__device__ __forceinline__ Vec8 load8(const void* p, int64_t vec) {
  return widen<T>(load_raw<T>(p, vec));
}

template <typename T>
__device__ __forceinline__ void store8(void* p, int64_t vec, const Vec8& a) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(a.v[2 * i], a.v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    reinterpret_cast<uint4*>(p)[vec] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* q = reinterpret_cast<float4*>(p) + 2 * vec;
    q[0] = make_float4(a.v[0], a.v[1], a.v[2], a.v[3]);
    q[1] = make_float4(a.v[4], a.v[5], a.v[6], a.v[7]);
  }
}

// The weight's eight entries of a vec, in fp32.
__device__ __forceinline__ Vec8 load_weight(const void* g, int f32, int64_t vec) {
  return f32 ? load8<float>(g, vec) : load8<__nv_bfloat16>(g, vec);
}

// Sums of NV values over the block, in a fixed order.  One barrier: `buf`
// alternates between calls, so a slow warp may still read the other half.
template <int NV>
__device__ __forceinline__ void block_sums(float (&v)[NV], float* buf, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (warps == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) buf[i * kMaxNormWarps + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += buf[i * kMaxNormWarps + w];
    v[i] = s;
  }
}

// a / 448 rounded to nearest, from 1 / 448 in two parts (hi rounded down): a hi + a lo is within 2^-46 of the quotient
// before its one rounding, and a quotient by 7 lies 1/14 of a unit or more from a boundary, if it is not one of the numbers.
__device__ __forceinline__ float over_448(float a) {
  constexpr float kHi = 0x1.249248p-9f, kLo = 0x1.24924ap-33f;
  return __fmaf_rn(a, kHi, __fmul_rn(a, kLo));
}

// y / s for two values per instruction, with 1 / s = hi + lo.  hi is the hardware's reciprocal taken down by 2^-22, more than
// its error, so that lo > 0 and a quotient of -0 keeps its sign; with e = 1 - s hi, lo = hi (e + e^2).  y lo + y hi is
// within 2^-43 of the quotient before its one rounding, so it rounds as the quotient does unless that lies within
// 2^-19 units of a boundary.  y (448 / amax) is one rounding more, and at a midpoint of e4m3 that is a whole step
// of y8.  16,384 rows of 2560, in a graph: 61.6 us (61.7 with y (448 / amax), 62.1 with the reciprocal and the scale rounded by
// the compiler's functions, 63.6 with a step along the remainder y - t s, 7 more with a division each).  An infinite
// scale leaves 0 for what is finite, as a division does; above a scale of 1e30 lo is subnormal and has fewer bits.
struct Quotient {
  uint64_t hi, lo;
  __device__ __forceinline__ static uint64_t twice(float f) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(f));
    return r;
  }
  __device__ __forceinline__ explicit Quotient(float s) {
    const float r = rcp_fast(s) * (1.0f - 0x1p-22f), e = __fmaf_rn(-s, r, 1.0f);
    hi = twice(r);
    lo = twice(r > 0.0f ? __fmaf_rn(e, e, e) * r : 0.0f);
  }
  __device__ __forceinline__ float2 of(float y0, float y1) const {
    float2 o;
    asm("{\n\t.reg .b64 y, t;\n\tmov.b64 y, {%2, %3};\n\tmul.rn.f32x2 t, y, %5;\n\t"
        "fma.rn.f32x2 t, y, %4, t;\n\tmov.b64 {%0, %1}, t;\n\t}"
        : "=f"(o.x), "=f"(o.y)
        : "f"(y0), "f"(y1), "l"(hi), "l"(lo));
    return o;
  }
};

struct NormParams {
  const void* x;
  const void* res;
  const void* g;
  void* res_out;
  void* y;            // bf16, or null
  uint8_t* y8;        // e4m3, or null
  float* scales;      // [N, groups]
  int64_t N;
  int nvec;           // d / 8
  int groups;         // ceil(d / 128)
  int g_f32;
  float inv_d, eps;
};

struct NoRes {};

// A block per row; thread t holds the vecs t, t + T, ... of the row.  T is a
// multiple of 32, so a scale group is 16 neighbouring lanes.  Blocks that stay
// and walk over rows, the weight in registers, read no faster and left some SMs
// a row more than others (65,536 rows of 2048: 270 us, a block per row 238).
template <typename XT, typename RT, int C>
__global__ void __launch_bounds__(C == 1 ? 512 : kMaxNormThreads) rms_norm_kernel(const NormParams p) {
  constexpr bool kRes = !std::is_same<RT, NoRes>::value;
  __shared__ float buf[kMaxNormWarps];
  const int T = blockDim.x, warps = T >> 5;
  const int64_t row = blockIdx.x;
  const int64_t base = row * p.nvec;
  Vec8 h[C];
  Vec8 g[C];
  float ss[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int v = threadIdx.x + c * T;
    if (v < p.nvec) {
      h[c] = load8<XT>(p.x, base + v);
      if constexpr (kRes) {
        const Vec8 r = load8<RT>(p.res, base + v);
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[c].v[i] += r.v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) h[c].v[i] = 0.0f;
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int v = threadIdx.x + c * T;
    if (v < p.nvec) g[c] = load_weight(p.g, p.g_f32, v);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) ss[0] = fmaf(h[c].v[i], h[c].v[i], ss[0]);
    if constexpr (kRes) {
      const int v = threadIdx.x + c * T;
      if (p.res_out && v < p.nvec) store8<RT>(p.res_out, base + v, h[c]);
    }
  }
  block_sums<1>(ss, buf, warps);
  const float r = rsqrtf(fmaf(ss[0], p.inv_d, p.eps));
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int v = threadIdx.x + c * T;
    const bool in = v < p.nvec;
    Vec8 y;
#pragma unroll
    for (int i = 0; i < kVec; ++i) y.v[i] = in ? h[c].v[i] * r * g[c].v[i] : 0.0f;
    if (p.y && in) store8<__nv_bfloat16>(p.y, base + v, y);
    if (p.y8) {
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) a = fmaxf(a, fabsf(y.v[i]));
#pragma unroll
      for (int o = kGroupVecs / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      a = fmaxf(a, kAmaxMin);
      const float s = over_448(a);
      const Quotient by(s);
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* e = y.v + 4 * i;
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(by.of(e[0], e[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(by.of(e[2], e[3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
      }
      if (in) {
        reinterpret_cast<uint2*>(p.y8)[base + v] = make_uint2(w[0], w[1]);
        if (v % kGroupVecs == 0) p.scales[row * p.groups + v / kGroupVecs] = s;
      }
    }
  }
}

// ---- gradient -------------------------------------------------------------
//
//   xh = h r, t = gy g:   gx = r (t - xh m) + gres,   m = mean(t xh) = r (sum t h) / d
//   gg = sum over rows of gy xh
//
// xh and m stay near 1 and |t| whatever the size of h; r^3, in h r^3 (sum t h) / d, leaves fp32's
// range for |h| above 1e13 and, where eps allows it, below 1e-13.
//
// Both row sums (h^2 and t h) are reduced together; the block's share of gg
// stays in registers over its rows and goes to one row of the workspace, and
// a second kernel adds those rows in a fixed order: no atomics, the same bits
// on every run.

struct NormGradParams {
  const void* gy;
  const void* h;
  const void* g;
  const void* gres;
  void* gx;
  float* part;        // [gridDim.x, d], or null: no weight gradient
  int64_t N;
  int nvec, g_f32;
  float inv_d, eps;
};

//
// The next row's inputs are loaded before this row is reduced, and both rows
// stay as they lie in memory until they are used: with each row's loads behind
// the last one's barrier 16,384 rows of 2560 (bf16, gres) took 101 us, with both
// rows held in fp32 89, so 57.5.
template <typename GT, typename HT, int C, bool kRes, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 256 ? 2 : 1) rms_norm_grad_kernel(const NormGradParams p) {
  constexpr bool kAhead = kThreads <= 512;      // rows above 8192 columns: no registers for a second one
  __shared__ float buf[2][2 * kMaxNormWarps];
  const int T = blockDim.x, warps = T >> 5;
  Vec8 g[C], gg[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int v = threadIdx.x + c * T;
#pragma unroll
    for (int i = 0; i < kVec; ++i) g[c].v[i] = gg[c].v[i] = 0.0f;
    if (v < p.nvec) g[c] = load_weight(p.g, p.g_f32, v);
  }
  Raw8<HT> h[C], a[kRes ? C : 1], nh[C], na[kRes ? C : 1];
  Raw8<GT> t[C], nt[C];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int v = threadIdx.x + c * T;
      if (v < p.nvec) {
        nh[c] = load_raw<HT>(p.h, row * p.nvec + v);
        nt[c] = load_raw<GT>(p.gy, row * p.nvec + v);
        if constexpr (kRes) na[c] = load_raw<HT>(p.gres, row * p.nvec + v);
      }
    }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    nh[c] = Raw8<HT>{};
    nt[c] = Raw8<GT>{};
    if constexpr (kRes) na[c] = Raw8<HT>{};
  }
  if (kAhead && blockIdx.x < p.N) fetch(blockIdx.x);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x, flip ^= 1) {
    const int64_t base = row * p.nvec;
    float s[2] = {0.0f, 0.0f};
    if constexpr (!kAhead) fetch(row);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      h[c] = nh[c];
      t[c] = nt[c];
      if constexpr (kRes) a[c] = na[c];
    }
    if (kAhead && row + gridDim.x < p.N) fetch(row + gridDim.x);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Vec8 hv = widen<HT>(h[c]), tv = widen<GT>(t[c]);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        s[0] = fmaf(hv.v[i], hv.v[i], s[0]);
        s[1] = fmaf(tv.v[i] * g[c].v[i], hv.v[i], s[1]);
      }
    }
    block_sums<2>(s, buf[flip], warps);
    const float r = rsqrtf(fmaf(s[0], p.inv_d, p.eps));
    const float m = r * (s[1] * p.inv_d);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int v = threadIdx.x + c * T;
      if (v < p.nvec) {
        const Vec8 hv = widen<HT>(h[c]), tv = widen<GT>(t[c]);
        Vec8 o;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float xh = hv.v[i] * r;
          gg[c].v[i] = fmaf(tv.v[i], xh, gg[c].v[i]);
          o.v[i] = fmaf(-xh, m, tv.v[i] * g[c].v[i]) * r;
        }
        if constexpr (kRes) {
          const Vec8 av = widen<HT>(a[c]);
#pragma unroll
          for (int i = 0; i < kVec; ++i) o.v[i] += av.v[i];
        }
        store8<HT>(p.gx, base + v, o);
      }
    }
  }
  if (p.part) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int v = threadIdx.x + c * T;
      if (v < p.nvec) store8<float>(p.part, static_cast<int64_t>(blockIdx.x) * p.nvec + v, gg[c]);
    }
  }
}

// gg[c] = sum of the `rows` partial rows: a block per 32 columns, 32 rows at a time.
__global__ void __launch_bounds__(1024) norm_weight_sum_kernel(const float* part, int rows, int d, float* gg) {
  __shared__ float buf[32][33];
  pdl_wait();
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (col < d)
#pragma unroll 4
    for (int r = threadIdx.y; r < rows; r += 32) s += part[static_cast<int64_t>(r) * d + col];
  buf[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < d) {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += buf[r][threadIdx.x];
    gg[col] = t;
  }
}

// Vecs per thread and threads per row.
struct RowPlan {
  int c, threads;
};
// One vec each while a block's threads suffice: 16,384 rows of 2560 take the
// norm 62 us at one, 71 at two.  The gradient keeps a row and the next one in
// flight and rather has two (57.6 us, 63.5 at one) unless there are few rows
// (1100: 10.8 us with the weight's sum, 10.1 at one; 2000: 13.8 and 13.3).
RowPlan row_plan(int nvec, int64_t N, bool grad) {
  RowPlan rp;
  rp.c = nvec > 512 || (grad && nvec > 64 && N > 1024) ? 2 : 1;
  rp.threads = ((nvec + rp.c - 1) / rp.c + 31) / 32 * 32;
  return rp;
}

constexpr int kNormGradBlocksPerSm = 6;
constexpr int kKnownDevices = 16;        // devices whose answers are kept; others are asked every time

unsigned row_grid(int64_t N, int threads, int per_sm) {
  const int fit = 2048 / threads;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * (fit < per_sm ? fit : per_sm);
  return static_cast<unsigned>(N < cap ? N : cap);
}

template <typename XT, typename RT>
void launch_norm_c(const NormParams& p, cudaStream_t s) {
  const RowPlan rp = row_plan(p.nvec, p.N, false);
  const unsigned grid = static_cast<unsigned>(p.N);
  if (rp.c == 1) rms_norm_kernel<XT, RT, 1><<<grid, rp.threads, 0, s>>>(p);
  else rms_norm_kernel<XT, RT, 2><<<grid, rp.threads, 0, s>>>(p);
}

template <typename XT>
void launch_norm_x(const NormParams& p, int res_type, cudaStream_t s) {
  if (!p.res) launch_norm_c<XT, NoRes>(p, s);
  else if (res_type == KOLIBRI_TYPE_BF16) launch_norm_c<XT, __nv_bfloat16>(p, s);
  else launch_norm_c<XT, float>(p, s);
}

// One wave: as many blocks as are resident at once, at most `grid`, which is set to what was launched.  The number per SM
// is asked for once per device and block size (of this kernel); host threads that ask at once store the same answer.
template <typename GT, typename HT, int C, bool kRes, int kThreads>
cudaError_t launch_norm_grad_t(const NormGradParams& p, int threads, unsigned& grid, cudaStream_t s) {
  static std::atomic<int> known[kKnownDevices][kMaxNormThreads / 32 + 1];
  auto kern = rms_norm_grad_kernel<GT, HT, C, kRes, kThreads>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::atomic<int>* const slot = dev < kKnownDevices ? &known[dev][threads / 32] : nullptr;
  int n = slot ? slot->load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0);
    if (err != cudaSuccess) return err;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (slot) slot->store(n, std::memory_order_relaxed);
  }
  const unsigned most = static_cast<unsigned>(n * device_sm_count());
  if (grid > most) grid = most;
  kern<<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename GT, typename HT, bool kRes>
cudaError_t launch_norm_grad_c(const NormGradParams& p, const RowPlan& rp, unsigned& grid, cudaStream_t s) {
  if (rp.c == 1) return launch_norm_grad_t<GT, HT, 1, kRes, 512>(p, rp.threads, grid, s);
  if (rp.threads <= 256) return launch_norm_grad_t<GT, HT, 2, kRes, 256>(p, rp.threads, grid, s);
  if (rp.threads <= 512) return launch_norm_grad_t<GT, HT, 2, kRes, 512>(p, rp.threads, grid, s);
  return launch_norm_grad_t<GT, HT, 2, kRes, kMaxNormThreads>(p, rp.threads, grid, s);
}
template <typename GT, typename HT>
cudaError_t launch_norm_grad_r(const NormGradParams& p, const RowPlan& rp, unsigned& grid, cudaStream_t s) {
  return p.gres ? launch_norm_grad_c<GT, HT, true>(p, rp, grid, s) : launch_norm_grad_c<GT, HT, false>(p, rp, grid, s);
}

}  // namespace

cudaError_t launch_rms_norm(const void* x, int x_type, const void* res, int res_type, const void* weight,
                            int weight_type, float eps, int64_t N, int32_t d, void* res_out, void* y,
                            void* y8, float* scales, cudaStream_t s) {
  NormParams p{};
  p.x = x;
  p.res = res;
  p.g = weight;
  p.res_out = res_out;
  p.y = y;
  p.y8 = static_cast<uint8_t*>(y8);
  p.scales = scales;
  p.N = N;
  p.nvec = d / kVec;
  p.groups = (d + 127) / 128;
  p.g_f32 = weight_type == KOLIBRI_TYPE_F32;
  p.inv_d = 1.0f / static_cast<float>(d);
  p.eps = eps;
  if (x_type == KOLIBRI_TYPE_BF16) launch_norm_x<__nv_bfloat16>(p, res_type, s);
  else launch_norm_x<float>(p, res_type, s);
  return cudaGetLastError();
}

size_t rms_norm_grad_ws_bytes(int64_t N, int32_t d) {
  const RowPlan rp = row_plan(d / kVec, N, true);
  return sizeof(float) * static_cast<size_t>(row_grid(N, rp.threads, kNormGradBlocksPerSm)) * d;
}

cudaError_t launch_rms_norm_grad(const void* gy, int gy_type, const void* h, int h_type,
                                 const void* weight, int weight_type, float eps, const void* gres,
                                 int64_t N, int32_t d, void* gx, float* gweight, void* ws,
                                 cudaStream_t s) {
  NormGradParams p{};
  p.gy = gy;
  p.h = h;
  p.g = weight;
  p.gres = gres;
  p.gx = gx;
  p.part = gweight ? static_cast<float*>(ws) : nullptr;
  p.N = N;
  p.nvec = d / kVec;
  p.g_f32 = weight_type == KOLIBRI_TYPE_F32;
  p.inv_d = 1.0f / static_cast<float>(d);
  p.eps = eps;
  const RowPlan rp = row_plan(p.nvec, N, true);
  unsigned grid = row_grid(N, rp.threads, kNormGradBlocksPerSm);      // as the workspace was sized, at most
  cudaError_t err;
  if (gy_type == KOLIBRI_TYPE_BF16) {
    if (h_type == KOLIBRI_TYPE_BF16) err = launch_norm_grad_r<__nv_bfloat16, __nv_bfloat16>(p, rp, grid, s);
    else err = launch_norm_grad_r<__nv_bfloat16, float>(p, rp, grid, s);
  } else {
    if (h_type == KOLIBRI_TYPE_BF16) err = launch_norm_grad_r<float, __nv_bfloat16>(p, rp, grid, s);
    else err = launch_norm_grad_r<float, float>(p, rp, grid, s);
  }
  if (err != cudaSuccess || !gweight) return err;
  return launch_pdl(norm_weight_sum_kernel, dim3((d + 31) / 32), dim3(32, 32), 0, s, dim3(0, 0, 0),
                    static_cast<const float*>(p.part), static_cast<int>(grid), static_cast<int>(d), gweight);
}

}  // namespace kolibri
