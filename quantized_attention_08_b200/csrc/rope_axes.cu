// rope_axes.cu -- rotary positions with several axes (time, height, width)
// for Q and K in one launch.
//
// Rotation pair i turns by theta = pos[axis(i)] * inv_freq[i].  Far positions
// lose their angle in fp32 (near 10^6 radians a step of fp32 is 1/16 radian),
// so the angle is formed and reduced to half turns in fp64 -- a handful of
// operations per (token, pair), shared by all heads -- and only the reduced
// angle is rounded to fp32.  The rotation itself is the fused pre-pass's: fp32 products, then
// the sum, each rounded to nearest, one rounding to the tensor's type.
//
// Bound by HBM: every element is read once and written once.  A thread owns
// eight pairs (16 channels) of one token, keeps their cosines and sines in
// registers and walks over the heads, so that the angles cost little beside
// the traffic and no table exists.  Few heads share them less: of the measured copy
// rate 16 + 16 heads reach 0.92 (d 128, 400 to 540 MB each), 8 + 8 0.90, 4 + 1 0.84,
// 1 + 1 0.61.
#include <stdint.h>

#include <algorithm>

#include "serve_internal.h"
#include "serve_math.cuh"

namespace sage {

constexpr int kRopeThreads = 256;
// Heads loaded before the first is rotated: 2 heads take 88 us on H 16 + 16, N
// 32768, d 128, fp16 (537 MB: 0.93 of the measured copy rate), 1 97, 4 93.
constexpr int kRopeUnroll = 2;

// x cos - y sin and y cos + x sin, each product and each sum rounded once
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = a;
}

// plain loads: the output may be the input
__device__ __forceinline__ uint4 rope_ld(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) k_rope_axes(RopeArgs a, int heads_per_cta) {
  after_previous();
  const int units = a.d / 16;  // threads a token
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / units) + threadIdx.x / units;
  const int u = threadIdx.x % units;
  if (item >= static_cast<int64_t>(a.B) * a.N) return;
  const int b = static_cast<int>(item / a.N), n = static_cast<int>(item % a.N);

  // channels of this thread: two runs of eight, at c0 and c1
  const int rot = a.pairs / 8;  // units that rotate; the others pass through
  const bool turns = u < rot;
  const int c0 = turns ? (INTERLEAVED ? 16 * u : 8 * u) : 2 * a.pairs + 16 * (u - rot);
  const int c1 = turns && !INTERLEAVED ? a.pairs + 8 * u : c0 + 8;

  float cs[8], sn[8];
  if (turns) {
    const int32_t* pos = a.pos + b * a.pos_s[1] + n;
    double p[kMaxAxes];
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) p[x] = x < a.axes ? static_cast<double>(pos[x * a.pos_s[0]]) : 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = 8 * u + e;
      double at = p[0];
#pragma unroll
      for (int x = 1; x < kMaxAxes; ++x)
        if (x < a.axes && i >= a.sec_end[x - 1]) at = p[x];
      // half turns: theta / pi, less an even whole number
      const double h = at * static_cast<double>(a.inv_freq[i]) * 0.31830988618379067154;
      const float r = static_cast<float>(h - 2.0 * rint(0.5 * h));
      sincospif(r, &sn[e], &cs[e]);
    }
  }

  const int h0 = blockIdx.y * heads_per_cta;
  const int h1 = min(a.heads[0] + a.heads[1], h0 + heads_per_cta);
  for (int hh = h0; hh < h1; hh += kRopeUnroll) {
    uint4 lo[kRopeUnroll], hi[kRopeUnroll];
#pragma unroll
    for (int j = 0; j < kRopeUnroll; ++j) {
      if (hh + j >= h1) break;
      const int w = hh + j >= a.heads[0];
      const int h = hh + j - (w ? a.heads[0] : 0);
      const T* src = static_cast<const T*>(a.in[w]) + b * a.in_s[w][0] + h * a.in_s[w][1] + n * a.in_s[w][2];
      lo[j] = rope_ld(src + c0);
      hi[j] = rope_ld(src + c1);
    }
#pragma unroll
    for (int j = 0; j < kRopeUnroll; ++j) {
      if (hh + j >= h1) break;
      const int w = hh + j >= a.heads[0];
      const int h = hh + j - (w ? a.heads[0] : 0);
      uint32_t x[4] = {lo[j].x, lo[j].y, lo[j].z, lo[j].w};
      uint32_t y[4] = {hi[j].x, hi[j].y, hi[j].z, hi[j].w};
      if (turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 p = unpack16<T>(x[e]), q = unpack16<T>(y[e]);
          if (INTERLEAVED) {  // pairs are neighbours: e and 4 + e
            turn(p.x, p.y, cs[e], sn[e]);
            turn(q.x, q.y, cs[4 + e], sn[4 + e]);
          } else {
            turn(p.x, q.x, cs[2 * e], sn[2 * e]);
            turn(p.y, q.y, cs[2 * e + 1], sn[2 * e + 1]);
          }
          x[e] = pack16<T>(p.x, p.y);
          y[e] = pack16<T>(q.x, q.y);
        }
      }
      T* dst = static_cast<T*>(a.out[w]) + b * a.out_s[w][0] + h * a.out_s[w][1] + n * a.out_s[w][2];
      *reinterpret_cast<uint4*>(dst + c0) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(dst + c1) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

cudaError_t launch_rope_axes(const RopeArgs& a, cudaStream_t st) {
  const int tokens_per_cta = kRopeThreads / (a.d / 16);
  const int64_t items = static_cast<int64_t>(a.B) * a.N;
  const int64_t gx = (items + tokens_per_cta - 1) / tokens_per_cta;
  const int heads = a.heads[0] + a.heads[1];
  // All heads in one CTA when the tokens alone fill the GPU a few times over;
  // fewer heads a CTA otherwise, down to one unrolled group.
  const int want = static_cast<int>(std::min<int64_t>((4 * kSms + gx - 1) / gx, (heads + kRopeUnroll - 1) / kRopeUnroll));
  const int hpc = ((heads + want - 1) / want + kRopeUnroll - 1) / kRopeUnroll * kRopeUnroll;
  const dim3 grid(static_cast<unsigned>(gx), (heads + hpc - 1) / hpc);
  auto* f = a.bf16 ? (a.interleaved ? k_rope_axes<__nv_bfloat16, true> : k_rope_axes<__nv_bfloat16, false>)
                   : (a.interleaved ? k_rope_axes<__half, true> : k_rope_axes<__half, false>);
  return launch_after(f, grid, kRopeThreads, 0, st, 1, a, hpc);
}

}  // namespace sage
