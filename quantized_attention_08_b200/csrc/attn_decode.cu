// attn_decode.cu -- attention of one new token, or a few, over a paged
// key-value cache, split over the cache's length and joined.
//
//   s_t = sm_scale * q . k_t,  k_t = code_t * delta_K[t]      (or 16-bit k_t)
//   m = max s, l = sum exp(s_t - m), o = sum exp(s_t - m) v_t / l
//
// Bound by HBM: each visible key and value is read once and serves all G
// query heads of its group (and all query tokens).
//
// Work.  The cache of one (request, kv head, group of query rows) is a
// segment of steps of kStep tokens.  All segments' steps stand in one line,
// and every warp of the grid takes an equal stretch of it, whatever the
// lengths: a long request is split over many warps, short ones share one.
// The lengths stay on the device; each CTA forms their prefix sum.  A segment
// inside one warp's stretch is finished there; the pieces of the others go to
// the workspace as (m, l, o) and a second kernel joins them in a fixed order.
//
// Loads.  One lane of a warp feeds the warp's own ring in shared memory with
// bulk copies of whole rows (a step of a page is one run of memory for each of
// K, V and the scales), counted by an mbarrier a stage; no other warp is
// involved.  cp.async by the lanes that later read the bytes, in fragment order,
// reached 4.9 TB/s where rows in order reach 6.5 (eight lanes then touch two
// to four lines at once).
//
// Products.  mma.sync m16n8k16, transposed: S^T = K q^T and O^T = V^T P^T,
// with tokens (channels) on the 16 side and query rows on the 8 side, since
// one token's group has 1 to 8 rows; 16 rows a tile would compute twice as
// much for nothing.  The tcgen05 form has 128 rows at least; at one to eight
// rows the tensor work here is a few percent of what HBM leaves time for.
// The order of k inside the products is free, so a lane's 16-byte pieces of
// K's rows serve as fragments as they are; pairs of V's rows are interleaved
// with prmt.  int8 codes become 16-bit numbers exactly; delta_K multiplies the
// fp32 scores, delta_V the probabilities.  S, m, l, O are fp32; P is rounded
// to 16 bits for its product (2^-12 or 2^-9 relative, as every 16-bit
// attention does), l sums the unrounded values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "sage_ptx.cuh"
#include "serve_internal.h"

namespace sage {

namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kMaxBatch = 4096;   // prefix sums in shared memory
constexpr int kSms = 148;
constexpr int kMinSteps = 2;      // of one warp's stretch

struct DecodeParams {
  const uint8_t* q;
  int64_t q_s[3];
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  int64_t k_page, v_page;        // bytes
  int64_t ks_page, vs_page;      // elements
  const int32_t* table;
  const int32_t* lens;
  uint8_t* o;
  float* lse;
  float* part_o;                 // [2 * workers][rows of a group][D]
  float2* part_ml;               // [2 * workers][rows of a group]
  int* prefix;                   // [B + 1] steps before each request
  int num_pages, page_size, max_pages;
  int B, H, Hk, G, n_q, rows, groups;  // rows = G * n_q in `groups` groups of 8 NT
  int max_len, causal, workers;
  float scale_log2;
  uint64_t timeout_ns;
};

// ------------------------------------------------------------ types
template <typename T>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t bytes(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}

// Four int8 codes as four 16-bit numbers, exactly.
//  fp16: 1024 + (code + 128) is the bit pattern 0x64 followed by the biased
//        byte; subtracting 1152 leaves the code.
//  bf16: 128 + (low seven bits) is 0x43 followed by them, and 0x43 followed by
//        the top bit alone is 128 or 256; the difference is the code.
template <typename T>
__device__ __forceinline__ void codes_to_16(uint32_t w, uint32_t& lo, uint32_t& hi);
template <>
__device__ __forceinline__ void codes_to_16<__half>(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  uint32_t x = bytes(u, 0x64646464u, 0x4140), y = bytes(u, 0x64646464u, 0x4342);
  const __half2 a = __hsub2(*reinterpret_cast<__half2*>(&x), bias);
  const __half2 b = __hsub2(*reinterpret_cast<__half2*>(&y), bias);
  lo = *reinterpret_cast<const uint32_t*>(&a);
  hi = *reinterpret_cast<const uint32_t*>(&b);
}
template <>
__device__ __forceinline__ void codes_to_16<__nv_bfloat16>(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t m = w & 0x7f7f7f7fu, s = w & 0x80808080u;
  uint32_t x0 = bytes(m, 0x43434343u, 0x4140), x1 = bytes(m, 0x43434343u, 0x4342);
  uint32_t y0 = bytes(s, 0x43434343u, 0x4140), y1 = bytes(s, 0x43434343u, 0x4342);
  const __nv_bfloat162 a = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x0), *reinterpret_cast<__nv_bfloat162*>(&y0));
  const __nv_bfloat162 b = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x1), *reinterpret_cast<__nv_bfloat162*>(&y1));
  lo = *reinterpret_cast<const uint32_t*>(&a);
  hi = *reinterpret_cast<const uint32_t*>(&b);
}

// Four E4M3 codes of token t (word a) and of token t' (word b), as four pairs
// (t, t') of 16-bit numbers, exactly.
//  bf16: E4M3's exponent and mantissa bits, moved to the low end of bf16's
//        exponent and the top of its mantissa, read 2^-120 times the number
//        (its subnormals too).
template <typename T>
__device__ __forceinline__ void e4m3_pairs(uint32_t a, uint32_t b, uint32_t* out);
template <>
__device__ __forceinline__ void e4m3_pairs<__half>(uint32_t a, uint32_t b, uint32_t* out) {
  const uint32_t x = bytes(a, b, 0x5140), y = bytes(a, b, 0x7362);
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(out[0]), "=r"(out[1])
      : "r"(x));
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(out[2]), "=r"(out[3])
      : "r"(y));
}
template <>
__device__ __forceinline__ void e4m3_pairs<__nv_bfloat16>(uint32_t a, uint32_t b, uint32_t* out) {
  const __nv_bfloat162 up = __bfloat162bfloat162(__ushort_as_bfloat16(0x7b80));  // 2^120
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t y = bytes(a, b, 0x4400 + 0x1111 * i);
    uint32_t z = (y & 0x80008000u) | ((y >> 4) & 0x07f007f0u);
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&z), up);
    out[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bulk copy of n bytes (a multiple of 16; both addresses 16-byte aligned),
// counted by `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t n, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(n), "r"(smem_u32(bar))
               : "memory");
}

// -------------------------------------------------------- shapes of a step
template <int D, int FMT>
struct Step {
  static constexpr int KB = FMT == SAGE_KV_16 ? 2 : 1;   // bytes of a K element
  static constexpr int VB = FMT == SAGE_KV_8P8 ? 1 : 2;
  static constexpr int KROW = D * KB, VROW = D * VB;     // bytes of a row
  static constexpr int KC = KROW / 64;                   // 16-byte pieces of a lane's K row (4 lanes a row)
  static constexpr int VW = VROW / 8 < 16 ? 8 : 16;      // bytes of a lane's piece of a V row (8 lanes a row)
  static constexpr int VC = VROW / (8 * VW);
  static constexpr int VE = VW / VB;                     // channels of a piece
  static constexpr bool KS = FMT != SAGE_KV_16;
  static constexpr bool VS = FMT == SAGE_KV_8P8;
  // 16-token tiles of a step: about 8 KB a step
  static constexpr int SUB = D == 128 ? (FMT == SAGE_KV_8P8 ? 2 : 1) : (FMT == SAGE_KV_8P8 ? 4 : 2);
  static constexpr int TOK = 16 * SUB;
  // a stage of the ring: K rows, V rows, K scales, V scales
  static constexpr int V_AT = TOK * KROW;
  static constexpr int KS_AT = V_AT + TOK * VROW;
  static constexpr int VS_AT = KS_AT + (KS ? TOK * 4 : 0);
  static constexpr int STAGE = VS_AT + (VS ? TOK * 4 : 0);
  static constexpr int TOKEN = KROW + VROW + (KS ? 4 : 0) + (VS ? 4 : 0);  // bytes of a token
};

inline __host__ __device__ int steps_of(int len, int tok) { return (len + tok - 1) / tok; }

__device__ __forceinline__ int clamp_len(const DecodeParams& p, int len) {
  const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
  len = max(len, 0);
  len = min(len, p.max_len);
  return static_cast<int>(len < room ? len : room);
}

// Where a warp stands in the line of steps.
struct Cursor {
  int b, z, step, steps, len;
};

// ------------------------------------------------------------- the kernel
template <typename T, int D, int FMT, int NT, bool SPLIT>
__global__ void __launch_bounds__(kWarps * 32, 1) k_attn_decode(const DecodeParams p) {
  using S = Step<D, FMT>;
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_scan[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int HZ = p.Hk * p.groups;
  uint8_t* const ring = smem + warp * (kStages * S::STAGE);
  __shared__ __align__(8) uint64_t s_bar[kWarps][kStages];
  __shared__ int s_abort[kWarps];
  uint64_t* const bar = s_bar[warp];
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) mbar_init(bar + i, 1);
    s_abort[warp] = 0;
    fence_mbar_init();
  }
  __syncwarp();
  int* s_prefix = reinterpret_cast<int*>(smem + kWarps * kStages * S::STAGE);  // SPLIT only: [B + 1]

  // ---- this warp's stretch [at, end) of the line
  // warp-major numbers: few workers then stand on as many SMs as they can
  const int worker = warp * gridDim.x + blockIdx.x;
  int64_t at = 0, end = 0;
  Cursor cur;
  if (SPLIT) {
    int run = 0;
    for (int b0 = 0; b0 < p.B; b0 += kWarps * 32) {
      const int b = b0 + threadIdx.x;
      int v = b < p.B ? steps_of(clamp_len(p, p.lens[b]), S::TOK) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = v;
      __syncthreads();
      int before = run;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        run += s_scan[w];
      }
      if (b < p.B) s_prefix[b + 1] = before + v;
    }
    if (threadIdx.x == 0) s_prefix[0] = 0;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b <= p.B; b += kWarps * 32) p.prefix[b] = s_prefix[b];
    // the join's CTAs may be placed now; they wait for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t total = static_cast<int64_t>(s_prefix[p.B]) * HZ;
    const int64_t per = max(static_cast<int64_t>(kMinSteps), (total + p.workers - 1) / p.workers);
    at = worker * per;
    end = min(total, at + per);
    if (worker >= p.workers || at >= end) return;
    // the request that holds step `at`: the last one with prefix * HZ <= at
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<int64_t>(s_prefix[mid]) * HZ <= at) lo = mid; else hi = mid;
    }
    cur.b = lo;
    cur.steps = s_prefix[lo + 1] - s_prefix[lo];
    const int64_t in = at - static_cast<int64_t>(s_prefix[lo]) * HZ;
    cur.z = static_cast<int>(in / cur.steps);
    cur.step = static_cast<int>(in - static_cast<int64_t>(cur.z) * cur.steps);
    cur.len = clamp_len(p, p.lens[lo]);
  } else {
    if (worker >= p.B * HZ) return;
    cur.b = worker / HZ;
    cur.z = worker % HZ;
    cur.step = 0;
    cur.len = clamp_len(p, p.lens[cur.b]);
    cur.steps = steps_of(cur.len, S::TOK);
    end = cur.steps;
  }

  // ---- issue side
  Cursor iss = cur;
  int64_t iss_left = end - at;         // steps not issued yet
  int tile_page = 0, tile_off = 0;     // page index and offset in the page of the next tile
  int page_base = -1, page_ids = 0;    // lane i holds table[page_base + i]
  auto seek = [&]() {
    const int t = iss.step * S::TOK;
    tile_page = t / p.page_size;
    tile_off = t - tile_page * p.page_size;
    page_base = -1;
  };
  seek();

  uint32_t absent = 0;  // 4 bits a stage: tiles on no page
  // The page of the next tile; page tables are read 32 entries at a time.
  auto next_page = [&]() {
    if (page_base < 0 || tile_page >= page_base + 32) {
      page_base = tile_page;
      const int i = page_base + lane;
      page_ids = i < p.max_pages && static_cast<int64_t>(i) * p.page_size < iss.len
                     ? p.table[static_cast<int64_t>(iss.b) * p.max_pages + i]
                     : -1;
    }
    return __shfl_sync(0xffffffffu, page_ids, tile_page - page_base);
  };
  // Copies of n tokens from offset tile_off of `page` to row `at` of a stage.
  auto copy = [&](uint8_t* stage, uint64_t* b, int page, int at, int n) {
    const int64_t in_page = static_cast<int64_t>(iss.z / p.groups) * p.page_size + tile_off;
    const uint32_t dst = smem_u32(stage);
    bulk_load(dst + at * S::KROW, p.k + page * p.k_page + in_page * S::KROW, n * S::KROW, b);
    bulk_load(dst + S::V_AT + at * S::VROW, p.v + page * p.v_page + in_page * S::VROW, n * S::VROW, b);
    if (S::KS) bulk_load(dst + S::KS_AT + at * 4, p.ks + page * p.ks_page + in_page, n * 4, b);
    if (S::VS) bulk_load(dst + S::VS_AT + at * 4, p.vs + page * p.vs_page + in_page, n * 4, b);
  };
  auto issue = [&](int slot) {
    if (iss_left <= 0) return;
    uint8_t* const stage = ring + slot * S::STAGE;
    uint32_t gone = 0;
    if (p.page_size % S::TOK == 0) {  // a step lies in one page
      const int page = next_page();
      const bool good = page >= 0 && page < p.num_pages;
      if (!good) gone = (1u << S::SUB) - 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar + slot, good ? S::TOK * S::TOKEN : 0);
        if (good) copy(stage, bar + slot, page, 0, S::TOK);
      }
      tile_off += S::TOK;
      if (tile_off == p.page_size) {
        tile_off = 0;
        ++tile_page;
      }
    } else {
#pragma unroll
      for (int s = 0; s < S::SUB; ++s) {
        const bool in = iss.step * S::TOK + 16 * s < iss.len;
        const int page = in ? next_page() : -1;
        const bool good = page >= 0 && page < p.num_pages;
        if (!good) gone |= 1u << s;
        if (lane == 0) {
          // the last tile's arrival closes the stage's count
          const uint32_t n = good ? 16 * S::TOKEN : 0;
          if (s + 1 < S::SUB) mbar_expect_tx(bar + slot, n);
          else mbar_arrive_expect_tx(bar + slot, n);
          if (good) copy(stage, bar + slot, page, 16 * s, 16);
        }
        tile_off += 16;
        if (tile_off == p.page_size) {
          tile_off = 0;
          ++tile_page;
        }
      }
    }
    absent = (absent & ~(15u << 4 * slot)) | gone << 4 * slot;
    --iss_left;
    if (++iss.step == iss.steps && iss_left > 0) {  // on to the next segment
      iss.step = 0;
      if (++iss.z == HZ) {
        iss.z = 0;
        do {
          ++iss.b;
          iss.steps = s_prefix[iss.b + 1] - s_prefix[iss.b];
        } while (iss.steps == 0);
        iss.len = clamp_len(p, p.lens[iss.b]);
      }
      seek();
    }
  };

#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);

  // ---- consume side
  int slot = 0;
  uint32_t parity = 0;
  int64_t left = end - at;
  bool first_piece = true;
  do {
    // one piece: steps [cur.step, stop) of one segment
    const int stop = static_cast<int>(min(static_cast<int64_t>(cur.steps), cur.step + left));
    const bool whole = cur.step == 0 && stop == cur.steps;
    const int h = cur.z / p.groups, row0 = (cur.z % p.groups) * ROWS;

    // q as B fragments, its channels in the order of K's pieces
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + 8 * n + g;
      const bool in = r < p.rows;
      const int qi = in ? r / p.G : 0, hh = h * p.G + (in ? r - qi * p.G : 0);
      const T* src = reinterpret_cast<const T*>(p.q) + cur.b * p.q_s[0] + hh * p.q_s[1] + qi * p.q_s[2];
      constexpr int PER = 16 / S::KB;  // channels of a K piece
#pragma unroll
      for (int x = 0; x < S::KC; ++x)
#pragma unroll
        for (int y = 0; y < PER / 8; ++y) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (in) w = *reinterpret_cast<const uint4*>(src + x * 4 * PER + c * PER + 8 * y);
          const int ks = x * (PER / 4) + 2 * y;
          qf[n][ks][0] = w.x;
          qf[n][ks][1] = w.y;
          qf[n][ks + 1][0] = w.z;
          qf[n][ks + 1][1] = w.w;
        }
    }
    // keys visible to this lane's two rows of each tile
    int vis[NT][2];
    int vis_min = cur.len;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row0 + 8 * n + 2 * c + e;
        vis[n][e] = cur.len;
        if (p.causal && r < p.rows) vis[n][e] = cur.len - p.n_q + 1 + r / p.G;
      }
    if (p.causal) vis_min = cur.len - p.n_q + 1;

    float acc[NT][D / 16][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.f;
    }

    for (; cur.step < stop; ++cur.step, --left) {
      __syncwarp();  // every lane is done with the stage that is filled next
      {
        int next = slot + kStages - 1;
        if (next >= kStages) next -= kStages;
        issue(next);
      }
      uint8_t* const base = ring + slot * S::STAGE;
      const bool there = mbar_wait(bar + slot, parity, s_abort + warp, p.timeout_ns, 0xD0);
      if (!__all_sync(0xffffffffu, there)) {
        // Given up (the error word says so).  The copies under way write to this
        // CTA's memory: wait for them too, as long again at most.
        const uint64_t since = globaltimer();
        for (int64_t n = left; n > 0 && n > left - kStages; --n) {
          while (!mbar_try_wait_hint(bar + slot, parity) && globaltimer() - since < p.timeout_ns) {
          }
          if (++slot == kStages) {
            slot = 0;
            parity ^= 1;
          }
        }
        return;
      }
      const int t0 = cur.step * S::TOK;
      const uint32_t gone = absent >> 4 * slot & 15;
      if (++slot == kStages) {
        slot = 0;
        parity ^= 1;
      }
      // Behind the last token the page may hold anything, and a tile on no page
      // was not copied.  Their scores are masked below; their V is zeroed here,
      // since 0 * NaN would reach the sums.
      if (t0 + S::TOK > cur.len || gone != 0) {
#pragma unroll
        for (int u = 0; u < S::SUB; ++u) {
          const int have = gone >> u & 1 ? 0 : min(16, max(0, cur.len - t0 - 16 * u));
          for (int i = 16 * (have * (S::VROW / 16) + lane); i < 16 * S::VROW; i += 512)
            *reinterpret_cast<uint4*>(base + S::V_AT + 16 * u * S::VROW + i) = make_uint4(0, 0, 0, 0);
          if (S::VS && lane >= have && lane < 16)
            *reinterpret_cast<float*>(base + S::VS_AT + (16 * u + lane) * 4) = 0.f;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }

      // ---- scores, in units of log2
      float s[NT][S::SUB][4];
#pragma unroll
      for (int u = 0; u < S::SUB; ++u) {
        const uint8_t* const kb = base + (16 * u + g) * S::KROW + c * 16;
        float s2[NT][4];  // a second accumulator: two chains of products, half as long
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][u][e] = s2[n][e] = 0.f;
#pragma unroll
        for (int x = 0; x < S::KC; ++x) {
          const uint4 w0 = *reinterpret_cast<const uint4*>(kb + x * 64);
          const uint4 w1 = *reinterpret_cast<const uint4*>(kb + 8 * S::KROW + x * 64);
          const uint32_t a0[4] = {w0.x, w0.y, w0.z, w0.w}, a1[4] = {w1.x, w1.y, w1.z, w1.w};
          if (S::KB == 2) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t a[4] = {a0[2 * y], a1[2 * y], a0[2 * y + 1], a1[2 * y + 1]};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<T>(y ? s2[n] : s[n][u], a, qf[n][2 * x + y][0], qf[n][2 * x + y][1]);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t a[4];
              codes_to_16<T>(a0[y], a[0], a[2]);
              codes_to_16<T>(a1[y], a[1], a[3]);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816<T>(y & 1 ? s2[n] : s[n][u], a, qf[n][(4 * x + y) % (D / 16)][0],
                            qf[n][(4 * x + y) % (D / 16)][1]);
            }
          }
        }
        float f0 = p.scale_log2, f1 = p.scale_log2;
        if (S::KS) {
          const uint8_t* const sb = base + S::KS_AT + u * 64;
          f0 *= *reinterpret_cast<const float*>(sb + g * 4);
          f1 *= *reinterpret_cast<const float*>(sb + (g + 8) * 4);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          s[n][u][0] = (s[n][u][0] + s2[n][0]) * f0;
          s[n][u][1] = (s[n][u][1] + s2[n][1]) * f0;
          s[n][u][2] = (s[n][u][2] + s2[n][2]) * f1;
          s[n][u][3] = (s[n][u][3] + s2[n][3]) * f1;
        }
      }
      // ---- masks: the end of the cache, later query tokens' keys, bad pages
      if (t0 + S::TOK > vis_min || gone != 0) {
#pragma unroll
        for (int u = 0; u < S::SUB; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = t0 + 16 * u + g + 8 * (e >> 1);
              if (t >= vis[n][e & 1] || (gone >> u & 1)) s[n][u][e] = -INFINITY;
            }
      }
      // ---- running maxima: reduced over the lanes only when one grew
      bool grew = false;
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[n][0][e], s[n][0][e + 2]);
#pragma unroll
          for (int u = 1; u < S::SUB; ++u) t = fmaxf(t, fmaxf(s[n][u][e], s[n][u][e + 2]));
          top[n][e] = t;
          grew |= t > m[n][e];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = top[n][e];
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            t = fmaxf(t, m[n][e]);
            alpha[e] = t == m[n][e] ? 1.f : exp2_fast(m[n][e] - t);
            m[n][e] = t;
            l[n][e] *= alpha[e];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[n][i][0] *= alpha[0];
            acc[n][i][1] *= alpha[1];
            acc[n][i][2] *= alpha[0];
            acc[n][i][3] *= alpha[1];
          }
        }
      }
      // ---- probabilities and O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < S::SUB; ++u) {
        const uint8_t* const vb = base + S::V_AT + (16 * u + 2 * c) * S::VROW + g * S::VW;
        uint32_t pf[NT][2];
        float f0 = 1.f, f1 = 1.f;
        if (S::VS) {
          // fp16: times 448, i.e. the row's largest |v|, which fp16 can hold;
          // delta_V itself would push small rows into fp16's subnormals
          const float up = std::is_same<T, __half>::value ? 448.f : 1.f;
          const uint8_t* const sb = base + S::VS_AT + u * 64;
          f0 = *reinterpret_cast<const float*>(sb + g * 4) * up;
          f1 = *reinterpret_cast<const float*>(sb + (g + 8) * 4) * up;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
          float e0 = exp2_fast(s[n][u][0] - m0), e1 = exp2_fast(s[n][u][1] - m1);
          float e2 = exp2_fast(s[n][u][2] - m0), e3 = exp2_fast(s[n][u][3] - m1);
          l[n][0] += e0 + e2;
          l[n][1] += e1 + e3;
          if (S::VS) {
            e0 *= f0;
            e1 *= f0;
            e2 *= f1;
            e3 *= f1;
          }
          pf[n][0] = transpose8x8(pack16<T>(e0, e1));
          pf[n][1] = transpose8x8(pack16<T>(e2, e3));
        }
#pragma unroll
        for (int x = 0; x < S::VC; ++x) {
          if (S::VB == 2) {
            const uint8_t* const v0 = vb + x * 128;
            const uint4 r0 = *reinterpret_cast<const uint4*>(v0);
            const uint4 r1 = *reinterpret_cast<const uint4*>(v0 + S::VROW);
            const uint4 r2 = *reinterpret_cast<const uint4*>(v0 + 8 * S::VROW);
            const uint4 r3 = *reinterpret_cast<const uint4*>(v0 + 9 * S::VROW);
            const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
            const uint32_t w2[4] = {r2.x, r2.y, r2.z, r2.w}, w3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a[4] = {bytes(w0[i], w1[i], 0x5410), bytes(w0[i], w1[i], 0x7632),
                                     bytes(w2[i], w3[i], 0x5410), bytes(w2[i], w3[i], 0x7632)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<T>(acc[n][(4 * x + i) % (D / 16)], a, pf[n][0], pf[n][1]);
            }
          } else {
            uint32_t w[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint8_t* const v0 = vb + ((j & 1) + 8 * (j >> 1)) * S::VROW;
              if (S::VW == 16) {
                const uint4 r = *reinterpret_cast<const uint4*>(v0);
                w[j][0] = r.x;
                w[j][1] = r.y;
                w[j][2] = r.z;
                w[j][3] = r.w;
              } else {
                const uint2 r = *reinterpret_cast<const uint2*>(v0);
                w[j][0] = r.x;
                w[j][1] = r.y;
              }
            }
#pragma unroll
            for (int i = 0; i < S::VW / 4; ++i) {
              uint32_t x01[4], x23[4];
              e4m3_pairs<T>(w[0][i], w[1][i], x01);
              e4m3_pairs<T>(w[2][i], w[3][i], x23);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t a[4] = {x01[2 * y], x01[2 * y + 1], x23[2 * y], x23[2 * y + 1]};
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma16816<T>(acc[n][(2 * i + y) % (D / 16)], a, pf[n][0], pf[n][1]);
              }
            }
          }
        }
      }
    }

    // ---- end of the piece
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = l[n][e];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        l[n][e] = t;
      }
    const float down = S::VS && std::is_same<T, __half>::value ? 1.f / 448.f : 1.f;
    // Channels of a lane: VE neighbours of each of the VC pieces (a V piece's
    // channels are spread over VE / 2 tiles, two a tile).
    constexpr int TILES = S::VE / 2;
    if (!SPLIT || whole) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = row0 + 8 * n + 2 * c + e;
          if (r >= p.rows) continue;
          const int qi = r / p.G, hh = h * p.G + (r - qi * p.G);
          const int64_t out = (static_cast<int64_t>(cur.b) * p.H + hh) * p.n_q + qi;
          const float f = l[n][e] > 0.f ? down / l[n][e] : 0.f;
          T* dst = reinterpret_cast<T*>(p.o) + out * D + g * S::VE;
#pragma unroll
          for (int x = 0; x < S::VC; ++x)
#pragma unroll
            for (int i = 0; i < TILES; i += 4) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                w[y] = pack16<T>(acc[n][x * TILES + i + y][e] * f, acc[n][x * TILES + i + y][e + 2] * f);
              *reinterpret_cast<uint4*>(dst + x * 8 * S::VE + 2 * i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          if (p.lse != nullptr && g == 0)
            p.lse[out] = l[n][e] > 0.f ? (m[n][e] + log2f(l[n][e])) * 0.69314718055994531f : -INFINITY;
        }
    } else {
      const int64_t slot_p = 2 * static_cast<int64_t>(worker) + (first_piece ? 0 : 1);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * c + e;
          if (row0 + r >= p.rows) continue;
          float* dst = p.part_o + (slot_p * ROWS + r) * D + g * S::VE;
#pragma unroll
          for (int x = 0; x < S::VC; ++x)
#pragma unroll
            for (int i = 0; i < TILES; i += 2)
              *reinterpret_cast<float4*>(dst + x * 8 * S::VE + 2 * i) =
                  make_float4(acc[n][x * TILES + i][e] * down, acc[n][x * TILES + i][e + 2] * down,
                              acc[n][x * TILES + i + 1][e] * down, acc[n][x * TILES + i + 1][e + 2] * down);
          if (g == 0) p.part_ml[slot_p * ROWS + r] = make_float2(m[n][e], l[n][e]);
        }
    }
    first_piece = false;
    if (!SPLIT || left <= 0) break;
    cur.step = 0;
    if (++cur.z == HZ) {
      cur.z = 0;
      do {
        ++cur.b;
        cur.steps = s_prefix[cur.b + 1] - s_prefix[cur.b];
      } while (cur.steps == 0);
      cur.len = clamp_len(p, p.lens[cur.b]);
    }
  } while (true);
}

// ------------------------------------------------------------------ join
// One CTA per output row; its warps take the row's pieces in turn and are
// joined in the order of the warps, so the sum's order is fixed.  Rows of
// requests without tokens are zeros.
constexpr int kJoinWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attn_join(const DecodeParams p, int rows_per_group) {
  constexpr int PER = D / 32;
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int HZ = p.Hk * p.groups;
  // grid: x = row of the group, y = kv head and group, z = request
  const int r = blockIdx.x % p.rows, h = blockIdx.x / p.rows, b = blockIdx.y;
  const int group = r / rows_per_group;
  const int qi = r / p.G, hh = h * p.G + (r - qi * p.G);
  const int64_t out = (static_cast<int64_t>(b) * p.H + hh) * p.n_q + qi;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int steps = p.prefix[b + 1] - p.prefix[b];
  T* dst = reinterpret_cast<T*>(p.o) + out * D;
  if (steps == 0) {
    for (int i = threadIdx.x; i < D; i += kJoinWarps * 32) dst[i] = T(0.f);
    if (p.lse != nullptr && threadIdx.x == 0) p.lse[out] = -INFINITY;
    return;
  }
  const int64_t total = static_cast<int64_t>(p.prefix[p.B]) * HZ;
  const int64_t per = max(static_cast<int64_t>(kMinSteps), (total + p.workers - 1) / p.workers);
  const int64_t s0 = static_cast<int64_t>(p.prefix[b]) * HZ + static_cast<int64_t>(h * p.groups + group) * steps;
  const int64_t w0 = s0 / per, w1 = (s0 + steps - 1) / per;
  if (w0 == w1) return;  // one piece: finished where it was computed
  float m = -INFINITY, l = 0.f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  const int rg = r - group * rows_per_group;
  for (int64_t w = w0 + warp; w <= w1; w += kJoinWarps) {
    // a worker's first piece is in its first place, any other in its second
    const int64_t slot = 2 * w + (w == w0 && s0 != w0 * per ? 1 : 0);
    const float2 ml = p.part_ml[slot * rows_per_group + rg];
    const float* src = p.part_o + (slot * rows_per_group + rg) * D + lane * PER;
    float x[PER];
    if (PER == 4) {
      const float4 f = *reinterpret_cast<const float4*>(src);
      x[0] = f.x;
      x[1] = f.y;
      x[PER - 2] = f.z;
      x[PER - 1] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(src);
      x[0] = f.x;
      x[1] = f.y;
    }
    const float t = fmaxf(m, ml.x);
    if (t == -INFINITY) continue;  // nothing visible so far
    const float fa = exp2_fast(m - t), fb = exp2_fast(ml.x - t);
    l = l * fa + ml.y * fb;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = o[i] * fa + x[i] * fb;
    m = t;
  }
  if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
  for (int i = 0; i < PER; ++i) s_o[warp][lane * PER + i] = o[i];
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) mm = fmaxf(mm, s_ml[w].x);
  float ll = 0.f, a0 = 0.f, a1 = 0.f;
  if (mm != -INFINITY) {
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = exp2_fast(s_ml[w].x - mm);
      ll += s_ml[w].y * f;
      a0 += s_o[w][2 * threadIdx.x] * f;
      a1 += s_o[w][2 * threadIdx.x + 1] * f;
    }
  }
  const float f = ll > 0.f ? 1.f / ll : 0.f;
  reinterpret_cast<uint32_t*>(dst)[threadIdx.x] = pack16<T>(a0 * f, a1 * f);
  if (p.lse != nullptr && threadIdx.x == 0)
    p.lse[out] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994531f : -INFINITY;
}

// ---------------------------------------------------------------- the plan
// Everything the host decides, from sizes alone (the lengths are on the
// device): how many query rows a warp takes, whether segments are split, and
// how many workers share the line.
struct Plan {
  int nt, groups, step_tokens, workers, ctas;
  bool split;
  size_t off_ml, off_prefix, bytes;
};

int step_tokens(int d, int format) {
  const int sub = d == 128 ? (format == SAGE_KV_8P8 ? 2 : 1) : (format == SAGE_KV_8P8 ? 4 : 2);
  return 16 * sub;
}

Plan plan_of(int B, int H, int H_kv, int n_q, int d, int max_len, int format) {
  Plan P = {};
  const int rows = H / H_kv * n_q;
  P.nt = rows <= 8 ? 1 : 2;
  P.groups = (rows + 8 * P.nt - 1) / (8 * P.nt);
  P.step_tokens = step_tokens(d, format);
  const int64_t steps = steps_of(max_len, P.step_tokens);
  const int64_t segments = static_cast<int64_t>(B) * H_kv * P.groups;
  const int64_t most = static_cast<int64_t>(kSms) * kWarps;
  P.split = steps > 4;
  int64_t workers = P.split ? std::min(most, (segments * steps + kMinSteps - 1) / kMinSteps) : segments;
  P.workers = static_cast<int>(workers);
  P.ctas = static_cast<int>(P.split ? std::min<int64_t>(kSms, workers)
                                    : std::max<int64_t>(std::min<int64_t>(kSms, workers), (workers + kWarps - 1) / kWarps));
  if (P.split) {
    const size_t slots = 2 * static_cast<size_t>(workers) * 8 * P.nt;
    P.off_ml = slots * d * sizeof(float);
    P.off_prefix = P.off_ml + slots * sizeof(float2);
    P.bytes = (P.off_prefix + (static_cast<size_t>(B) + 1) * sizeof(int) + 255) / 256 * 256;
  }
  return P;
}

template <typename T, int D, int FMT, int NT, bool SPLIT>
cudaError_t launch_one(const DecodeParams& p, const Plan& P, cudaStream_t st) {
  using S = Step<D, FMT>;
  constexpr int kRing = kWarps * kStages * S::STAGE;
  const size_t smem = kRing + (SPLIT ? (static_cast<size_t>(p.B) + 1) * sizeof(int) : 0);
  auto* f = k_attn_decode<T, D, FMT, NT, SPLIT>;
  // always the same value: calls of other host threads may set it too
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kRing + (SPLIT ? (kMaxBatch + 1) * static_cast<int>(sizeof(int)) : 0));
  if (e != cudaSuccess) return e;
  f<<<P.ctas, kWarps * 32, smem, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess || !SPLIT) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows * p.Hk, p.B);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attn_join<T, D>, p, 8 * NT);
}

template <typename T, int D, int FMT>
cudaError_t launch_fmt(const DecodeParams& p, const Plan& P, cudaStream_t st) {
  if (P.nt == 1)
    return P.split ? launch_one<T, D, FMT, 1, true>(p, P, st) : launch_one<T, D, FMT, 1, false>(p, P, st);
  return P.split ? launch_one<T, D, FMT, 2, true>(p, P, st) : launch_one<T, D, FMT, 2, false>(p, P, st);
}
template <typename T, int D>
cudaError_t launch_d(const DecodeParams& p, const Plan& P, int format, cudaStream_t st) {
  if (format == SAGE_KV_16) return launch_fmt<T, D, SAGE_KV_16>(p, P, st);
  if (format == SAGE_KV_B) return launch_fmt<T, D, SAGE_KV_B>(p, P, st);
  return launch_fmt<T, D, SAGE_KV_8P8>(p, P, st);
}

}  // namespace

cudaError_t decode_read_and_clear_error(uint32_t* word) {
  uint32_t w = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&w, g_error_word, sizeof(w));
  if (e != cudaSuccess) return e;
  if (w != 0) e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
  *word = w;
  return e;
}

size_t decode_workspace_bytes(int B, int H, int H_kv, int n_q, int d, int max_len, int format) {
  return plan_of(B, H, H_kv, n_q, d, max_len, format).bytes;
}

cudaError_t launch_attn_decode(const DecodeArgs& a, cudaStream_t st) {
  const sage_kv_cache_t& c = a.c;
  const Plan P = plan_of(a.B, a.H, c.H_kv, a.n_q, c.d, a.max_len, c.format);
  DecodeParams p = {};
  p.q = static_cast<const uint8_t*>(a.q);
  for (int i = 0; i < 3; ++i) p.q_s[i] = a.q_s[i];
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.k_page = c.k_page_stride * (c.format == SAGE_KV_16 ? 2 : 1);
  p.v_page = c.v_page_stride * (c.format == SAGE_KV_8P8 ? 1 : 2);
  p.ks_page = c.k_scale_page_stride;
  p.vs_page = c.v_scale_page_stride;
  p.table = a.block_table;
  p.lens = a.seq_lens;
  p.o = static_cast<uint8_t*>(a.o);
  p.lse = a.lse;
  if (P.split) {
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + P.off_ml);
    p.prefix = reinterpret_cast<int*>(ws + P.off_prefix);
  }
  p.num_pages = c.num_pages;
  p.page_size = c.page_size;
  p.max_pages = a.max_pages;
  p.B = a.B;
  p.H = a.H;
  p.Hk = c.H_kv;
  p.G = a.H / c.H_kv;
  p.n_q = a.n_q;
  p.rows = p.G * a.n_q;
  p.groups = P.groups;
  p.max_len = c.num_pages > 0 ? a.max_len : 0;  // no page: no token
  p.causal = a.causal;
  p.workers = P.workers;
  p.timeout_ns = a.timeout_ns;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  if (c.dtype == SAGE_F16)
    return c.d == 64 ? launch_d<__half, 64>(p, P, c.format, st) : launch_d<__half, 128>(p, P, c.format, st);
  return c.d == 64 ? launch_d<__nv_bfloat16, 64>(p, P, c.format, st)
                   : launch_d<__nv_bfloat16, 128>(p, P, c.format, st);
}

}  // namespace sage
