// kvcache.cu -- the paged key-value cache: page tables and slot maps from
// request lengths, and the append that quantizes new tokens into their slots.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cooperative_groups.h>
#include <stdint.h>

#include <algorithm>

#include "quant_pair.cuh"
#include "serve_internal.h"

namespace sage {

namespace cg = cooperative_groups;

// ------------------------------------------------------------- k_kv_slots
// One launch, one cluster: every CTA forms the two prefix sums over the
// requests (new tokens, new pages) for itself in shared memory -- the lengths
// are a few KB in L2, cheaper to read again than to pass on -- and takes its
// share of the tokens and of the new pages.  Bound by latency: launch, one
// read of the lengths, two block scans, one dependent read (an old table
// entry or a free page), the stores.  The cluster barrier separates the last
// read of ctx_lens and free_used from the first write of seq_lens and
// free_used_out, so that these may be the same arrays (a captured step that
// is replayed).
constexpr int kSlotThreads = 1024;
constexpr int kSlotCtas = 8;  // portable cluster size
constexpr int kSlotMaxBatch = 8192;

// Inclusive scan of one value per thread over the block; *total gets the sum.
__device__ __forceinline__ long long block_scan(long long v, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // s_warp may still be read from the scan before
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  long long w = s_warp[lane];  // kSlotThreads / 32 == 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  const long long before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
  *total = __shfl_sync(0xffffffffu, w, 31);
  return v + (warp == 0 ? 0 : before);
}

// Last index b in [0, n) with a[b] <= i (a non-decreasing, a[0] <= i).  Of a
// run of equal entries it is the last, so requests without tokens are passed.
__device__ __forceinline__ int find_owner(const int* a, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kSlotThreads) k_kv_slots(SlotArgs a) {
  extern __shared__ int s_slots[];
  int* s_cu = s_slots;               // [B + 1] first token of each request
  int* s_first = s_cu + a.B + 1;     // [B + 1] first new page of each request
  int* s_ctx = s_first + a.B + 1;    // [B] cached tokens
  __shared__ long long s_warp[32];

  const int P = a.page_size;
  const int room = a.max_pages * P;  // < 2^31 (checked by the caller)
  int used = *a.free_used;
  used = min(max(used, 0), a.num_free);

  if (threadIdx.x == 0) s_cu[0] = s_first[0] = 0;
  // first tokens, cut to [0, T]
  long long run = 0;
  for (int b0 = 0; b0 < a.B; b0 += kSlotThreads) {
    const int b = b0 + threadIdx.x;
    int ctx = 0, n = 0;
    if (b < a.B) {
      ctx = min(max(a.ctx_lens[b], 0), room);
      n = min(max(a.new_lens[b], 0), room - ctx);
    }
    long long total;
    const long long incl = run + block_scan(n, s_warp, &total);
    if (b < a.B) {
      s_ctx[b] = ctx;
      s_cu[b + 1] = static_cast<int>(incl < a.T ? incl : a.T);
    }
    run += total;
  }
  __syncthreads();
  // first new pages
  run = 0;
  for (int b0 = 0; b0 < a.B; b0 += kSlotThreads) {
    const int b = b0 + threadIdx.x;
    int need = 0;
    if (b < a.B) {
      const int ctx = s_ctx[b], end = ctx + (s_cu[b + 1] - s_cu[b]);
      need = static_cast<int>((static_cast<unsigned>(end) + P - 1) / P - (static_cast<unsigned>(ctx) + P - 1) / P);
    }
    long long total;
    const long long incl = run + block_scan(need, s_warp, &total);
    if (b < a.B) {
      s_first[b + 1] = static_cast<int>(incl);
    }
    run += total;
  }
  __syncthreads();
  const int rank = blockIdx.x, ctas = gridDim.x;
  if (ctas > 1) cg::this_cluster().sync();

  const int have = a.num_free - used;  // pages left in the free list
  const int wanted = s_first[a.B];
  if (rank == 0) {
    for (int b = threadIdx.x; b <= a.B; b += kSlotThreads) {
      a.cu_seqlens[b] = s_cu[b];
      if (b == a.B) break;
      const int ctx = s_ctx[b], end = ctx + (s_cu[b + 1] - s_cu[b]);
      const int held = static_cast<int>((static_cast<unsigned>(ctx) + P - 1) / P);
      const int got = min(s_first[b + 1] - s_first[b], max(0, have - s_first[b]));
      const long long backed = static_cast<long long>(held + got) * P;
      a.seq_lens[b] = static_cast<int>(end < backed ? end : backed);
    }
    if (threadIdx.x == 0) *a.free_used_out = used + min(wanted, have);
  }
  const int step = ctas * kSlotThreads;
  for (int i = rank * kSlotThreads + threadIdx.x; i < wanted; i += step) {
    const int b = find_owner(s_first, a.B, i);
    const int held = static_cast<int>((static_cast<unsigned>(s_ctx[b]) + P - 1) / P);
    a.block_table[static_cast<size_t>(b) * a.max_pages + held + (i - s_first[b])] =
        i < have ? a.free_pages[used + i] : -1;
  }
  const int tokens = s_cu[a.B];
  for (int i = rank * kSlotThreads + threadIdx.x; i < a.T; i += step) {
    int slot = -1, pos = -1, b = -1;
    if (i < tokens) {
      b = find_owner(s_cu, a.B, i);
      pos = s_ctx[b] + (i - s_cu[b]);
      const int held = static_cast<int>((static_cast<unsigned>(s_ctx[b]) + P - 1) / P);
      const int pi = pos / P;
      int page;
      if (pi < held) {
        page = a.block_table[static_cast<size_t>(b) * a.max_pages + pi];
      } else {
        const int at = s_first[b] + (pi - held);
        page = at < have ? a.free_pages[used + at] : -1;
      }
      // a page whose slots would pass 2^31 is no page of any cache
      if (page >= 0 && page <= (0x7fffffff - P) / P) slot = page * P + (pos - pi * P);
    }
    a.slot_map[i] = slot;
    a.positions[i] = pos;
    a.seq_ids[i] = b;
  }
}

cudaError_t launch_kv_slots(const SlotArgs& a, cudaStream_t st) {
  const size_t smem = (3 * static_cast<size_t>(a.B) + 2) * sizeof(int);
  if (smem > 32 * 1024) {
    static OncePerDevice once;
    const cudaError_t e = once.run([&] {
      return cudaFuncSetAttribute(k_kv_slots, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (3 * kSlotMaxBatch + 2) * static_cast<int>(sizeof(int)));
    });
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  // one CTA serves a decode step without the cluster barrier
  cfg.gridDim = dim3(a.T <= kSlotThreads && a.B <= kSlotThreads ? 1 : kSlotCtas);
  cfg.blockDim = dim3(kSlotThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cfg.gridDim.x;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv_slots, a);
}

// ------------------------------------------------------------ k_kv_append
// Per (token, kv head) row: K minus the request's channel means (Smooth K:
// softmax does not change when every key of a request moves by one vector),
// then int8 codes with one scale per row, delta = max|x| / 127; V as E4M3
// with delta = max|v| / 448, or unchanged.  A scale per token, because a
// cache grows: a scale per 128-token block or per channel, as the prefill
// uses, would change with every token that joins.  Bound by HBM: each input
// is read once and each code written once.  Two lanes' worth of channels a
// thread (channels 8c.. and d/2 + 8c..), so that a row takes d / 16 lanes and
// its maximum log2(d / 16) shuffles.
constexpr int kAppendThreads = 256;
constexpr float kTinyScale = 7.88860905e-31f;  // 2^-100

template <typename T>
__device__ __forceinline__ float2 to_f2(uint32_t w);
template <>
__device__ __forceinline__ float2 to_f2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 to_f2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t from_f2(float2 f);
template <>
__device__ __forceinline__ uint32_t from_f2<__half>(float2 f) {
  const __half2 h = __float22half2_rn(f);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t from_f2<__nv_bfloat16>(float2 f) {
  const __nv_bfloat162 h = __float22bfloat162_rn(f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// maximum over the LANES lanes that share a row
template <int LANES>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// delta = RN(top * step), step = RN(1 / 127) or RN(1 / 448): a scale within
// one ulp of top / range, so that |x| / delta <= range (1 + 2^-22) still
// rounds to the range's top.  0 where its reciprocal would leave fp32's normal
// numbers (only bf16 inputs, or all-zero rows, get there).
__device__ __forceinline__ float scale_of(float top, float step) {
  const float delta = __fmul_rn(top, step);
  return delta < kTinyScale ? 0.f : delta;
}

// E4M3 codes of 4 values (RN(x / delta), the sign of a zero kept)
__device__ __forceinline__ uint32_t e4m3_codes4(const float* x, float delta, float r) {
  const uint64_t nd2 = f2_pack(-delta, -delta), r2 = f2_pack(r, r);
  float2 a = f2_unpack(div2_rn(f2_pack(x[0], x[1]), nd2, r2));
  float2 b = f2_unpack(div2_rn(f2_pack(x[2], x[3]), nd2, r2));
  a.x = copysignf(a.x, x[0]);
  a.y = copysignf(a.y, x[1]);
  b.x = copysignf(b.x, x[2]);
  b.y = copysignf(b.y, x[3]);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(AppendArgs a, int rows_per_cta) {
  constexpr int LANES = D / 16;                  // threads a row
  constexpr int RPI = kAppendThreads / LANES;    // rows an iteration
  const int c = threadIdx.x % LANES;
  const int h = blockIdx.y;
  const int t0 = blockIdx.x * rows_per_cta;
  const int t1 = min(a.T, t0 + rows_per_cta);
  const int P = a.c.page_size;
  const int slots = a.c.num_pages * P;  // < 2^31 (checked by the caller)
  const T* kin = static_cast<const T*>(a.in[0]) + h * a.in_s[0][0] + 8 * c;
  const T* vin = static_cast<const T*>(a.in[1]) + h * a.in_s[1][0] + 8 * c;

  for (int base = t0; base < t1; base += RPI) {
    // every lane of the warp runs the loop: the row maxima are shuffles
    const int t = base + threadIdx.x / LANES;
    int slot = t < t1 ? a.slot_map[t] : -1;
    int seq = 0;
    if (a.mean_k != nullptr && t < t1) {
      seq = a.seq_ids[t];
      if (seq < 0 || seq >= a.B) slot = -1;
    }
    const bool live = slot >= 0 && slot < slots;
    uint4 k[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (live) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        k[i] = ld_once(kin + t * a.in_s[0][1] + i * (D / 2));
        v[i] = ld_once(vin + t * a.in_s[1][1] + i * (D / 2));
      }
    }
    const int page = live ? slot / P : 0;
    const int at = live ? slot - page * P : 0;
    const size_t row = static_cast<size_t>(h) * P + at;
    uint8_t* kout = static_cast<uint8_t*>(a.c.k);
    uint8_t* vout = static_cast<uint8_t*>(a.c.v);

    // ---- K
    float x[16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {k[i].x, k[i].y, k[i].z, k[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = to_f2<T>(w[e]);
        x[8 * i + 2 * e] = f.x;
        x[8 * i + 2 * e + 1] = f.y;
      }
    }
    if (a.mean_k != nullptr && live) {
      const float* m = a.mean_k + (static_cast<size_t>(seq) * a.c.H_kv + h) * D + 8 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 f = *reinterpret_cast<const float4*>(m + i * (D / 2) + 4 * e);
          x[8 * i + 4 * e] = __fsub_rn(x[8 * i + 4 * e], f.x);
          x[8 * i + 4 * e + 1] = __fsub_rn(x[8 * i + 4 * e + 1], f.y);
          x[8 * i + 4 * e + 2] = __fsub_rn(x[8 * i + 4 * e + 2], f.z);
          x[8 * i + 4 * e + 3] = __fsub_rn(x[8 * i + 4 * e + 3], f.w);
        }
    }
    if (FMT == SAGE_KV_16) {
      if (live) {
        uint8_t* p = kout + (page * a.c.k_page_stride + row * D + 8 * c) * sizeof(T);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint4 o = k[i];
          if (a.mean_k != nullptr)
            o = make_uint4(from_f2<T>(make_float2(x[8 * i], x[8 * i + 1])),
                           from_f2<T>(make_float2(x[8 * i + 2], x[8 * i + 3])),
                           from_f2<T>(make_float2(x[8 * i + 4], x[8 * i + 5])),
                           from_f2<T>(make_float2(x[8 * i + 6], x[8 * i + 7])));
          *reinterpret_cast<uint4*>(p + i * (D / 2) * sizeof(T)) = o;
        }
      }
    } else {
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
      const float delta = scale_of(row_max<LANES>(top), 1.f / 127.f);
      const float r = __frcp_rn(delta);
      const uint64_t nd2 = f2_pack(-delta, -delta), r2 = f2_pack(r, r);
      if (live) {
        uint8_t* p = kout + page * a.c.k_page_stride + row * D + 8 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint2 o = make_uint2(0, 0);
          if (delta != 0.f) {
            o.x = codes4(f2_pack(x[8 * i], x[8 * i + 1]), f2_pack(x[8 * i + 2], x[8 * i + 3]), nd2, r2);
            o.y = codes4(f2_pack(x[8 * i + 4], x[8 * i + 5]), f2_pack(x[8 * i + 6], x[8 * i + 7]), nd2, r2);
          }
          *reinterpret_cast<uint2*>(p + i * (D / 2)) = o;
        }
        if (c == 0) a.c.k_scale[page * a.c.k_scale_page_stride + row] = delta;
      }
    }

    // ---- V
    if (FMT != SAGE_KV_8P8) {
      if (live) {
        uint8_t* p = vout + (page * a.c.v_page_stride + row * D + 8 * c) * sizeof(T);
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(p + i * (D / 2) * sizeof(T)) = v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = to_f2<T>(w[e]);
          x[8 * i + 2 * e] = f.x;
          x[8 * i + 2 * e + 1] = f.y;
        }
      }
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
      const float delta = scale_of(row_max<LANES>(top), 1.f / 448.f);
      const float r = __frcp_rn(delta);
      if (live) {
        uint8_t* p = vout + page * a.c.v_page_stride + row * D + 8 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint2 o = make_uint2(0, 0);
          if (delta != 0.f) {
            o.x = e4m3_codes4(x + 8 * i, delta, r);
            o.y = e4m3_codes4(x + 8 * i + 4, delta, r);
          }
          *reinterpret_cast<uint2*>(p + i * (D / 2)) = o;
        }
        if (c == 0) a.c.v_scale[page * a.c.v_scale_page_stride + row] = delta;
      }
    }
  }
}

template <typename T, int D>
cudaError_t append_as(const AppendArgs& a, cudaStream_t st) {
  constexpr int RPI = kAppendThreads / (D / 16);
  const int rows = 2 * RPI;
  const dim3 grid((a.T + rows - 1) / rows, a.c.H_kv);
  if (a.c.format == SAGE_KV_16)
    k_kv_append<T, D, SAGE_KV_16><<<grid, kAppendThreads, 0, st>>>(a, rows);
  else if (a.c.format == SAGE_KV_B)
    k_kv_append<T, D, SAGE_KV_B><<<grid, kAppendThreads, 0, st>>>(a, rows);
  else
    k_kv_append<T, D, SAGE_KV_8P8><<<grid, kAppendThreads, 0, st>>>(a, rows);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
  if (a.c.dtype == SAGE_F16)
    return a.c.d == 64 ? append_as<__half, 64>(a, st) : append_as<__half, 128>(a, st);
  return a.c.d == 64 ? append_as<__nv_bfloat16, 64>(a, st) : append_as<__nv_bfloat16, 128>(a, st);
}

}  // namespace sage
