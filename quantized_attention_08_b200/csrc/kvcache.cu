// kvcache.cu -- the paged key-value cache: page tables and slot maps from
// request lengths, and the append that quantizes new tokens into their slots.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cooperative_groups.h>
#include <stdint.h>

#include <algorithm>

#include "quant_pair.cuh"
#include "serve_internal.h"
#include "serve_math.cuh"

namespace sage {

namespace cg = cooperative_groups;

// ------------------------------------------------------------- k_kv_slots
// One launch: every CTA forms the two prefix sums over the requests (new
// tokens, new pages) for itself in shared memory -- the lengths are a few KB in
// L2, cheaper to read again than to pass on -- and takes its share of the tokens
// and of the new pages.  Bound by latency: launch, one read of the lengths, two
// block scans, one dependent read (an old table entry or a free page), the
// stores.  Where seq_lens is ctx_lens or free_used_out is free_used (a captured
// step that is replayed), the CTAs are one cluster, whose barrier separates the
// last read of the old values from the first write of the new ones; eight CTAs at
// most then, which many places show: 256 places 3.5 us, in place 3.6; 4096 3.4 and
// 4.2; 65536 3.9 and 15.0.
constexpr int kSlotThreads = 512;
constexpr int kSlotCluster = 8;  // portable
constexpr int kSlotMaxBatch = 8192;
constexpr uint32_t kSlotCap = 1u << 30;  // of a sum of tokens: T is at most this

// Inclusive scan of one value per thread over the block, saturating at kSlotCap
// (values and sums up to it, so that two of them fit 32 bits); *total gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* s_warp, uint32_t* total) {
  constexpr int kSlotWarps = kSlotThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = min(v + u, kSlotCap);
  }
  __syncthreads();  // s_warp may still be read from the scan before
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  uint32_t w = lane < kSlotWarps ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 1; o < kSlotWarps; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w = min(w + u, kSlotCap);
  }
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
  *total = __shfl_sync(0xffffffffu, w, kSlotWarps - 1);
  return warp == 0 ? v : min(v + before, kSlotCap);
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

__global__ void __launch_bounds__(kSlotThreads) k_kv_slots(SlotArgs a, bool cluster) {
  extern __shared__ int s_slots[];
  int* s_cu = s_slots;               // [B + 1] first token of each request
  int* s_first = s_cu + a.B + 1;     // [B + 1] first new page of each request
  int* s_ctx = s_first + a.B + 1;    // [B] cached tokens
  __shared__ uint32_t s_warp[32];

  after_previous();
  const int P = a.page_size;
  const int room = a.max_pages * P;  // < 2^31 (checked by the caller)
  int used = *a.free_used;
  used = min(max(used, 0), a.num_free);

  if (threadIdx.x == 0) s_cu[0] = s_first[0] = 0;
  // first tokens, cut to [0, T]
  uint32_t run = 0;
  for (int b0 = 0; b0 < a.B; b0 += kSlotThreads) {
    const int b = b0 + threadIdx.x;
    int ctx = 0, n = 0;
    if (b < a.B) {
      ctx = min(max(a.ctx_lens[b], 0), room);
      n = min(max(a.new_lens[b], 0), room - ctx);
    }
    uint32_t total;
    const uint32_t incl = min(run + block_scan(min(static_cast<uint32_t>(n), kSlotCap), s_warp, &total), kSlotCap);
    if (b < a.B) {
      s_ctx[b] = ctx;
      s_cu[b + 1] = min(static_cast<int>(incl), a.T);
    }
    run = min(run + total, kSlotCap);
  }
  __syncthreads();
  // first new pages (at most one a token)
  run = 0;
  for (int b0 = 0; b0 < a.B; b0 += kSlotThreads) {
    const int b = b0 + threadIdx.x;
    uint32_t need = 0;
    if (b < a.B) {
      const unsigned ctx = s_ctx[b], end = ctx + (s_cu[b + 1] - s_cu[b]);
      need = (end + P - 1) / P - (ctx + P - 1) / P;
    }
    uint32_t total;
    const uint32_t incl = run + block_scan(need, s_warp, &total);
    if (b < a.B) s_first[b + 1] = static_cast<int>(incl);
    run += total;
  }
  __syncthreads();
  // in place: every CTA has read the old values
  if (cluster) cg::this_cluster().sync();
  const int rank = blockIdx.x, ctas = gridDim.x;

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
  const int64_t items = std::max<int64_t>(a.T, a.B);  // there are at most as many new pages
  const bool in_place = a.seq_lens == a.ctx_lens || a.free_used_out == a.free_used;
  const int ctas = static_cast<int>(std::min<int64_t>(std::max<int64_t>(1, (items + kSlotThreads - 1) / kSlotThreads),
                                                      in_place ? kSlotCluster : kSms));
  const int cluster = in_place ? ctas : 1;
  return launch_after(k_kv_slots, dim3(ctas), kSlotThreads, smem, st, cluster, a, cluster > 1);
}

// ------------------------------------------------------------ k_kv_append
// Per (token, kv head) row: K minus the request's channel means (Smooth K:
// softmax does not change when every key of a request moves by one vector),
// then int8 codes with one scale per row, delta = max|x| / 127; V as E4M3
// with delta = max|v| / 448, or unchanged.  A scale per token, because a
// cache grows: a scale per 128-token block or per channel, as the prefill
// uses, would change with every token that joins.
//
// Bound by HBM: each input is read once and each code written once.  A thread
// holds channels 8c .. and d/2 + 8c .. of a row, so that a row takes d / 16
// lanes and its maximum log2(d / 16) shuffles; its loads do not wait for its
// slot (a skipped token is read for nothing).  One row a thread and six CTAs an
// SM: 65536 tokens of 8 heads, d 128, fp16 with means, 8+8 (407 MB) take 67 us on the
// device, 0.93 of the measured copy rate (69 to 73 in sequence, where the power cap
// lowers the clock); two or four rows a thread with the next one's loads in flight
// took 9 and 27% longer (more registers, fewer warps).
constexpr int kAppendThreads = 256;

template <typename T>
__device__ __forceinline__ uint64_t to_f2(uint32_t w);  // the two values of w as fp32 (exact)
template <>
__device__ __forceinline__ uint64_t to_f2<__half>(uint32_t w) {
  return f2_from_h2(w);
}
template <>
__device__ __forceinline__ uint64_t to_f2<__nv_bfloat16>(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t from_f2(uint64_t f) {
  const float2 x = f2_unpack(f);
  return pack16<T>(x.x, x.y);
}

__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// the largest magnitude of a row: of this thread's 16 values, then of the LANES
// lanes that share the row
template <int LANES>
__device__ __forceinline__ float row_max(const uint64_t* x) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = f2_unpack(x[i]);
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(f.x), "f"(f.y));
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

// delta = RN(top * step), step = RN(1 / 127) or RN(1 / 448): a scale within
// one ulp of top / range, so that |x| / delta <= range (1 + 2^-22) still
// rounds to the range's top.  0 where its reciprocal would leave fp32's normal
// numbers (only bf16 inputs, or all-zero rows, get there).
__device__ __forceinline__ float scale_of(float top, float step) {
  const float delta = __fmul_rn(top, step);
  return delta < kTinyScale ? 0.f : delta;
}

// E4M3 codes of 4 values (RN(x / delta); a zero of either sign is code 0)
__device__ __forceinline__ uint32_t e4m3_codes4(uint64_t x01, uint64_t x23, uint64_t nd2, uint64_t r2) {
  const float2 a = f2_unpack(div2_rn(x01, nd2, r2)), b = f2_unpack(div2_rn(x23, nd2, r2));
  uint32_t w;
  asm("{.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};}"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return w;
}

// x / P for 0 <= x < 2^31: umulhi(x, mul) >> shift, mul = ceil(2^(32 + shift) / P),
// shift = ceil(log2 P) - 1 (Granlund and Montgomery, "Division by invariant
// integers using multiplication", PLDI 1994)
struct PageDiv {
  uint32_t mul;
  int shift;
};

template <typename T, int D, int FMT, bool MEAN>
__global__ void __launch_bounds__(kAppendThreads, 6) k_kv_append(const AppendArgs a, const PageDiv div) {
  constexpr int LANES = D / 16;                  // threads a row
  after_previous();
  const int c = threadIdx.x % LANES;
  const int h = blockIdx.y;
  const int t = blockIdx.x * (kAppendThreads / LANES) + threadIdx.x / LANES;
  const int u = min(t, a.T - 1);  // every lane of a warp stays: the row maxima are shuffles
  const int P = a.c.page_size;
  const int slots = a.c.num_pages * P;  // < 2^31 (checked by the caller)
  const T* kin = static_cast<const T*>(a.in[0]) + h * a.in_s[0][0] + u * a.in_s[0][1] + 8 * c;
  const T* vin = static_cast<const T*>(a.in[1]) + h * a.in_s[1][0] + u * a.in_s[1][1] + 8 * c;

  const uint4 k0 = ld_once(kin), k1 = ld_once(kin + D / 2);
  const uint4 v0 = ld_once(vin), v1 = ld_once(vin + D / 2);
  const int slot = t < a.T ? a.slot_map[u] : -1;
  const int seq = MEAN ? a.seq_ids[u] : 0;
  const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
  const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  const bool known = !MEAN || (seq >= 0 && seq < a.B);
  const bool live = slot >= 0 && slot < slots && known;
  // read here, while K and V are on their way (a fifth longer otherwise)
  uint64_t mean[8];
  if (MEAN && known) {
    const float* m = a.mean_k + (static_cast<size_t>(seq) * a.c.H_kv + h) * D + 8 * c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(m + (i >> 1) * (D / 2) + 4 * (i & 1));
      mean[2 * i] = f2_pack(f.x, f.y);
      mean[2 * i + 1] = f2_pack(f.z, f.w);
    }
  }
  const int page = live ? static_cast<int>(__umulhi(slot, div.mul) >> div.shift) : 0;
  const size_t row = static_cast<size_t>(h) * P + (live ? slot - page * P : 0);
  uint8_t* kout = static_cast<uint8_t*>(a.c.k);
  uint8_t* vout = static_cast<uint8_t*>(a.c.v);

  // ---- K
  uint64_t x[8];
  if (FMT != SAGE_KV_16 || MEAN) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = to_f2<T>(kw[i]);
      if (MEAN) x[i] = f2_sub(x[i], mean[i]);
    }
  }
  if (FMT == SAGE_KV_16) {
    if (live) {
      uint8_t* p = kout + (page * a.c.k_page_stride + row * D + 8 * c) * sizeof(T);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = MEAN ? from_f2<T>(x[4 * i + e]) : kw[4 * i + e];
        *reinterpret_cast<uint4*>(p + i * (D / 2) * sizeof(T)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  } else {
    const float delta = scale_of(row_max<LANES>(x), 1.f / 127.f);
    const float r = __frcp_rn(delta);
    const uint64_t nd2 = f2_pack(-delta, -delta), r2 = f2_pack(r, r);
    if (live) {
      uint8_t* p = kout + page * a.c.k_page_stride + row * D + 8 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint2 o = make_uint2(codes4(x[4 * i], x[4 * i + 1], nd2, r2), codes4(x[4 * i + 2], x[4 * i + 3], nd2, r2));
        if (delta == 0.f) o = make_uint2(0, 0);
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
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4*>(p + i * (D / 2) * sizeof(T)) =
            make_uint4(vw[4 * i], vw[4 * i + 1], vw[4 * i + 2], vw[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f2<T>(vw[i]);
    const float delta = scale_of(row_max<LANES>(x), 1.f / 448.f);
    const float r = __frcp_rn(delta);
    const uint64_t nd2 = f2_pack(-delta, -delta), r2 = f2_pack(r, r);
    if (live) {
      uint8_t* p = vout + page * a.c.v_page_stride + row * D + 8 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint2 o = make_uint2(e4m3_codes4(x[4 * i], x[4 * i + 1], nd2, r2),
                             e4m3_codes4(x[4 * i + 2], x[4 * i + 3], nd2, r2));
        if (delta == 0.f) o = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(p + i * (D / 2)) = o;
      }
      if (c == 0) a.c.v_scale[page * a.c.v_scale_page_stride + row] = delta;
    }
  }
}

template <typename T, int D, int FMT>
cudaError_t append_fmt(const AppendArgs& a, cudaStream_t st) {
  constexpr int rows = kAppendThreads / (D / 16);
  const dim3 grid((a.T + rows - 1) / rows, a.c.H_kv);
  PageDiv div;
  div.shift = 31 - __builtin_clz(a.c.page_size - 1);  // page_size >= 16
  div.mul = static_cast<uint32_t>(((uint64_t(1) << (32 + div.shift)) + a.c.page_size - 1) / a.c.page_size);
  if (a.mean_k != nullptr) return launch_after(k_kv_append<T, D, FMT, true>, grid, kAppendThreads, 0, st, 1, a, div);
  return launch_after(k_kv_append<T, D, FMT, false>, grid, kAppendThreads, 0, st, 1, a, div);
}

template <typename T, int D>
cudaError_t append_as(const AppendArgs& a, cudaStream_t st) {
  if (a.c.format == SAGE_KV_16) return append_fmt<T, D, SAGE_KV_16>(a, st);
  if (a.c.format == SAGE_KV_B) return append_fmt<T, D, SAGE_KV_B>(a, st);
  return append_fmt<T, D, SAGE_KV_8P8>(a, st);
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
  if (a.c.dtype == SAGE_F16)
    return a.c.d == 64 ? append_as<__half, 64>(a, st) : append_as<__half, 128>(a, st);
  return a.c.d == 64 ? append_as<__nv_bfloat16, 64>(a, st) : append_as<__nv_bfloat16, 128>(a, st);
}

}  // namespace sage
