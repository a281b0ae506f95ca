// expert_fp8_decode.cu -- the 8-bit expert layer for a few tokens: two launches
// that stream each slot's weights once, without tiles of 128 rows.
//
// The formulas are those of expert_fp8.cu.  Bound by HBM: a slot (token and
// expert) reads 3 d F bytes of weights and does 6 d F operations on them, far
// below what any tile would need; what matters is how many loads are in flight
// on all SMs and that there are few launches.
//
//   gate/up   a block per (row, 8 units): 8 gate and 8 up rows of the weights,
//             k blocks dealt to eight warps; h in fp32
//   down      a block per (token, 16 columns): a warp per slot of the token; h is
//             put into e4m3 as it is loaded, the slots' outputs meet in shared
//             memory and leave as y: no outputs per expert, no third pass.  It is
//             launched while the first kernel runs, and has its weights on their
//             way when h is there
//
// The products run on the warp-level matrix instruction m16n8k32 (16 weight
// rows, 32 of k; one of the eight columns is used): converting both operands to
// fp32 for ordinary multiply-adds would take longer than the loads.  The order
// of k inside a block is free as long as both operands agree, so a lane loads
// 16 consecutive bytes of its rows and feeds them as four operand words.
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "launch.h"
#include "approx.cuh"
#include "common.cuh"
#include "pdl.cuh"

namespace kolibri {

namespace {

constexpr float kAmaxMin = 1e-30f;
constexpr float kE4m3Max = 448.0f;
constexpr int kUnits = 8;                // hidden units per gate/up block
// Eight warps of two or three k blocks: 13.5 us for the layer of one token (d =
// 2560, 6 of 384 experts and the shared one, in a graph), 15.3 with four, 19.3 with two.
constexpr int kUpWarps = 8;
constexpr int kCols = 16;                // output columns per down block
constexpr int kAhead = 2;                // k blocks of down weights loaded at once
constexpr int kMaxSlots = KOLIBRI_MAX_TOPK + 1;

// c += A (16 rows x 32 of k) * B (32 of k x 8), e4m3, fp32 accumulation.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 128 of k from two 16-byte pieces per row: lane l holds rows l / 4 (lo) and l
// / 4 + 8 (hi), bytes 16 (l % 4) on of each half; x likewise.
__device__ __forceinline__ void mma_block(float (&c)[4], const uint4 (&lo)[2], const uint4 (&hi)[2], const uint4 (&x)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    mma_e4m3(c, lo[i].x, hi[i].x, lo[i].y, hi[i].y, x[i].x, x[i].y);
    mma_e4m3(c, lo[i].z, hi[i].z, lo[i].w, hi[i].w, x[i].z, x[i].w);
  }
}

// Weights are read once: past L1, first to leave L2.
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

struct Decode {
  const uint8_t* x8;
  const float* xs;
  const int64_t* offsets;
  const int32_t* inv;
  const float* gates;
  const uint8_t* wgu;
  const float* sgu;
  const uint8_t* wd;
  const float* sd;
  const uint8_t* wgu_s;
  const float* sgu_s;
  const uint8_t* wd_s;
  const float* sd_s;
  float* h;                 // [N K (+ N), F], by grouped row
  __nv_bfloat16* y;
  int64_t NK;
  int d, F, E, K, shared;
};

// A slot of a token: its grouped row and expert (E: the shared one).  The
// row's place and all offsets are loaded together, the expert is the number of
// segments that begin at or before the row, less one.  A bad entry of inv is
// reported and gives row 0; the expert is in [0, E) whatever the offsets hold.
__device__ __forceinline__ void place_of(const Decode& p, int64_t t, int k, int64_t& row, int& e) {
  row = p.NK + t;
  e = p.E;
  if (k == p.K) return;
  constexpr int kPer = KOLIBRI_MAX_EXPERTS / 32;
  const int lane = threadIdx.x & 31;
  int64_t off[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) off[i] = lane + 32 * i < p.E ? __ldg(p.offsets + lane + 32 * i) : INT64_MAX;
  const int32_t q = __ldg(p.inv + t * p.K + k);
  const bool bad = q < 0 || q >= p.NK;
  if (bad) raise_status(kStatusBadInput);
  row = bad ? 0 : q;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) n += off[i] <= row ? 1 : 0;
  n = __reduce_add_sync(0xffffffffu, n);
  e = n > 0 ? n - 1 : 0;
}

// grid (F / 8, N, K + shared).  Offsets that do not run from 0 to N K without
// decreasing are reported.
__global__ void __launch_bounds__(32 * kUpWarps) expert_up_decode_kernel(const Decode p) {
  __shared__ float part[kUpWarps][2][kUnits];
  pdl_wait();
  pdl_trigger();           // the down projection may begin to load its weights
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.y;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int g = threadIdx.x; g <= p.E; g += 32 * kUpWarps) {
      const int64_t o = p.offsets[g];
      if ((g == 0 && o != 0) || (g == p.E && o != p.NK) || (g > 0 && p.offsets[g - 1] > o)) raise_status(kStatusBadInput);
    }
  int64_t row;
  int e;
  place_of(p, t, blockIdx.z, row, e);
  const int kblocks = p.d / 128;
  const int u0 = blockIdx.x * kUnits;
  const bool sh = e == p.E;
  const uint8_t* w = sh ? p.wgu_s : p.wgu + static_cast<int64_t>(e) * 2 * p.F * p.d;
  const float* s = sh ? p.sgu_s : p.sgu + static_cast<int64_t>(e) * (2 * p.F / 128) * kblocks;
  const uint8_t* wg = w + static_cast<int64_t>(u0 + (lane >> 2)) * p.d + (lane & 3) * 16;
  const uint8_t* wu = wg + static_cast<int64_t>(p.F) * p.d;
  const uint8_t* x = p.x8 + t * p.d + (lane & 3) * 16;
  const float* sg = s + (u0 / 128) * kblocks;
  const float* su = sg + (p.F / 128) * kblocks;
  const float* xs = p.xs + t * kblocks;
  float g = 0.0f, u = 0.0f;              // column 0 of the accumulators: lanes 4 r hold units r
#pragma unroll 2
  for (int kb = warp; kb < kblocks; kb += kUpWarps) {
    uint4 a[2], b[2], xv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = load_stream(wg + kb * 128 + 64 * i);
      b[i] = load_stream(wu + kb * 128 + 64 * i);
      xv[i] = lane < 4 ? __ldg(reinterpret_cast<const uint4*>(x + kb * 128 + 64 * i)) : make_uint4(0, 0, 0, 0);
    }
    const float f = __ldg(xs + kb);
    float c[4] = {0.f, 0.f, 0.f, 0.f};
    mma_block(c, a, b, xv);
    g = fmaf(c[0], f * __ldg(sg + kb), g);
    u = fmaf(c[2], f * __ldg(su + kb), u);
  }
  if ((lane & 3) == 0) {
    part[warp][0][lane >> 2] = g;
    part[warp][1][lane >> 2] = u;
  }
  __syncthreads();
  if (threadIdx.x < kUnits) {
    float gs = 0.0f, us = 0.0f;
#pragma unroll
    for (int i = 0; i < kUpWarps; ++i) {
      gs += part[i][0][threadIdx.x];
      us += part[i][1][threadIdx.x];
    }
    p.h[row * p.F + u0 + threadIdx.x] = gs * rcp_fast(1.0f + exp2_fast(gs * -kLog2e)) * us;
  }
}

// grid (d / 16, N), a warp per slot of the token.  A lane holds the same 16
// bytes of k of every 64 as in the matrix operand, in fp32 from h; the maximum
// of a group of 128 is a maximum over the four lanes of a quad.
__global__ void __launch_bounds__(32 * kMaxSlots) expert_down_decode_kernel(const Decode p) {
  __shared__ float part[kMaxSlots][kCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.y;
  const int k = p.shared ? (warp == 0 ? p.K : warp - 1) : warp;      // the shared expert first, then k ascending
  int64_t row;
  int e;
  place_of(p, t, k, row, e);
  const int fblocks = p.F / 128;
  const int c0 = blockIdx.x * kCols;
  const bool sh = e == p.E;
  const uint8_t* w = (sh ? p.wd_s : p.wd + static_cast<int64_t>(e) * p.d * p.F) +
                     static_cast<int64_t>(c0 + (lane >> 2)) * p.F + (lane & 3) * 16;
  const float* s = (sh ? p.sd_s : p.sd + static_cast<int64_t>(e) * (p.d / 128) * fblocks) + (c0 / 128) * fblocks;
  const float* h = p.h + row * p.F + (lane & 3) * 16;
  float lo = 0.0f, hi = 0.0f;            // columns c0 + lane / 4 and + 8, in lanes 4 r
  for (int f0 = 0; f0 < fblocks; f0 += kAhead) {
    uint4 a[kAhead][2], b[kAhead][2];
    float sw[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (f0 + j < fblocks) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[j][i] = load_stream(w + (f0 + j) * 128 + 64 * i);
          b[j][i] = load_stream(w + static_cast<int64_t>(8) * p.F + (f0 + j) * 128 + 64 * i);
        }
        sw[j] = __ldg(s + f0 + j);
      }
    if (f0 == 0) pdl_wait();             // h; the inputs and weights loaded above are not written by the kernel before
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (f0 + j < fblocks) {
        const float4* hb = reinterpret_cast<const float4*>(h + (f0 + j) * 128);
        float4 v[8];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = hb[16 * (i / 4) + i % 4];
          m = fmaxf(m, fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2)), kAmaxMin);
        const float q = __fdiv_rn(kE4m3Max, m);
        uint4 hv[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t word[4];
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            const float4 f = v[4 * i + l];
            const uint32_t x01 = __nv_cvt_float2_to_fp8x2(make_float2(f.x * q, f.y * q), __NV_SATFINITE, __NV_E4M3);
            const uint32_t x23 = __nv_cvt_float2_to_fp8x2(make_float2(f.z * q, f.w * q), __NV_SATFINITE, __NV_E4M3);
            word[l] = lane < 4 ? x01 | (x23 << 16) : 0u;
          }
          hv[i] = make_uint4(word[0], word[1], word[2], word[3]);
        }
        const float f = __fdiv_rn(m, kE4m3Max) * sw[j];
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma_block(c, a[j], b[j], hv);
        lo = fmaf(c[0], f, lo);
        hi = fmaf(c[2], f, hi);
      }
  }
  if ((lane & 3) == 0) {
    const float gate = sh ? 1.0f : __ldg(p.gates + t * p.K + k);
    part[warp][lane >> 2] = lo * gate;
    part[warp][(lane >> 2) + 8] = hi * gate;
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
    float y = 0.0f;
    for (int i = 0; i < p.K + p.shared; ++i) y += part[i][threadIdx.x];
    p.y[t * p.d + c0 + threadIdx.x] = __float2bfloat16_rn(y);
  }
}

}  // namespace

bool expert_fp8_decode_preferred(int64_t N, int32_t K, bool shared) {
  return N * (K + (shared ? 1 : 0)) <= kFp8DecodeSlots;
}

cudaError_t launch_expert_ffn_fp8_decode(const ExpertFp8Args& a, cudaStream_t s) {
  Decode p{};
  p.x8 = static_cast<const uint8_t*>(a.x8);
  p.xs = a.x_scale;
  p.offsets = a.offsets;
  p.inv = a.inv;
  p.gates = a.gates;
  p.wgu = static_cast<const uint8_t*>(a.w_gate_up);
  p.sgu = a.s_gate_up;
  p.wd = static_cast<const uint8_t*>(a.w_down);
  p.sd = a.s_down;
  p.wgu_s = static_cast<const uint8_t*>(a.ws_gate_up);
  p.sgu_s = a.ss_gate_up;
  p.wd_s = static_cast<const uint8_t*>(a.ws_down);
  p.sd_s = a.ss_down;
  p.h = static_cast<float*>(a.ws);
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.NK = a.N * a.K;
  p.d = a.d;
  p.F = a.F;
  p.E = a.E;
  p.K = a.K;
  p.shared = a.ws_gate_up != nullptr ? 1 : 0;
  const unsigned slots = static_cast<unsigned>(a.K + p.shared), n = static_cast<unsigned>(a.N);
  cudaError_t err = launch_pdl(expert_up_decode_kernel, dim3(a.F / kUnits, n, slots), dim3(32 * kUpWarps), 0, s,
                               dim3(0, 0, 0), p);
  if (err != cudaSuccess) return err;
  return launch_pdl(expert_down_decode_kernel, dim3(a.d / kCols, n), dim3(32 * slots), 0, s, dim3(0, 0, 0), p);
}

KOLIBRI_DEFINE_STATUS_TAKE(status_take_expert_fp8_decode)

}  // namespace kolibri
