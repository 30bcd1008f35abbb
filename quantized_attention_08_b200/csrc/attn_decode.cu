// attn_decode.cu -- attention of one new token, or a few, over a paged
// key-value cache, split over the cache's length and joined.
//
//   s_t = sm_scale * q . k_t,  k_t = code_t * delta_K[t]      (or 16-bit k_t)
//   m = max s, l = sum exp(s_t - m), o = sum exp(s_t - m) v_t / l
//
// Bound by HBM: each visible key and value is read once and serves all G
// query heads of its group (and all query tokens).  Measured on one B200,
// device time with the join: 89 us for one request of 131072 tokens (H 32,
// H_kv 8, d 128, bf16: 537 MB, 0.92 of the measured copy rate), 93.4 us for 64
// requests of 1 to 8192 tokens in 8+8 (570 MB, 0.93; 96 to 103 us for seconds on end,
// when the power cap lowers the clock).
//
// Work.  The cache of one (request, kv head, group of query rows) is a
// segment of steps of S::TOK tokens.  All segments' steps stand in one line,
// and every consuming warp of the grid takes an equal stretch of it, whatever
// the lengths: a long request is split over many warps, short ones share one.
// The lengths stay on the device; each CTA forms their prefix sum.  A segment
// inside one warp's stretch is finished there; the pieces of the others go to
// the workspace as (m, l, o) and a second kernel joins them in a fixed order.
//
// Loads.  Loading warps feed a ring in shared memory for each consuming warp
// with bulk copies of whole rows (a step of a page is one run of memory for
// each of K, V and the scales), counted by an mbarrier a stage.  cp.async by the
// lanes that later read the bytes, in fragment order, reached 4.9 TB/s where
// rows in order reach 6.5 (eight lanes then touch two to four lines at once).
// A stage is released once K is multiplied and V is in registers.
//
// Products.  mma.sync m16n8k16, transposed: S^T = K q^T and O^T = V^T P^T,
// with tokens (channels) on the 16 side and query rows on the 8 side, since
// one token's group has 1 to 8 rows; 16 rows a tile would compute twice as
// much for nothing.  The tcgen05 forms have 64 rows at least; at one to sixteen
// the tensor pipe is 15 to 28 percent busy.
// The order of k inside the products is free, so a lane's 16-byte pieces of
// K's rows serve as fragments as they are; pairs of V's rows are interleaved
// with prmt.  int8 and E4M3 codes become fp16 numbers exactly; delta_K multiplies
// the fp32 scores, delta_V, in units of the largest one so far, the
// probabilities.  S, m, l, O are fp32.  P enters its product as two 16-bit numbers,
// its rounding and what that leaves, which is within 2^-16 of it.  For bf16 that is
// all; fp16 has few exponents, so P is taken in its upper range (2^10 or 2^11 is the
// largest when m is new), and where a P is so small that its second number would
// lose bits, a step's second numbers are taken 2^11 times as large and their sums
// put right.  What is lost then is at most 2^-47 of the largest P (with delta_V
// 2^-46 of the largest P times the largest delta_V).  One number instead of two
// made the output's error up to 1.5 times that of its own rounding, and lost the keys 17
// nats below the largest.  64 requests of 8+8 in sequence: 97.5 us fp16, 103 bf16 (99
// with one number); four drafted tokens, bf16: 43.1 (39.3).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "sage_ptx.cuh"
#include "serve_internal.h"
#include "serve_math.cuh"

namespace sage {

namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kFeeders = 4;   // loading warps
constexpr int kMaxBatch = 4096;   // prefix sums in shared memory
constexpr int kMinSteps = 2;      // of one warp's stretch
// How far scores may pass the running maximum before it follows (in log2).  With 0,
// some row of 8 or 16 grows in most steps of a stretch (four drafted tokens: 44.0 us;
// 39.3 with 4, 39.1 with 8, all with one number a P).  A larger one costs fp16 P its range.
constexpr float kSlack = 4.f;
// How many times the unit of O delta_V may be before it follows.
constexpr float kUnitSlack = 2.f;
// Where fp16 P stands (in log2): 2^15 is the largest it gets.
constexpr int kLift = 11, kLiftV = 10;
static_assert(kLift + kSlack == 15.f, "P, a score's lag included");
static_assert((1 << kLiftV) * kUnitSlack == (1 << kLift), "and P delta_V, the unit's included");
// of an instantiation; bf16 P needs none
__host__ __device__ constexpr int lift_of(bool half_p, int format) { return !half_p ? 0 : format == SAGE_KV_8P8 ? kLiftV : kLift; }
// How much larger the second numbers of small P are, and which are small: a number
// that is below fp16's normal ones is off by 2^-25, which is 2^-16 of 2^-9.  Below
// 2^-37 nothing of a P is left either way.
constexpr float kApart = 2048.f;
constexpr uint32_t kSmall = (127 - 9) << 23, kNothing = (127 - 37) << 23;  // as the bits of a float
// How the segments are spread over the warps.
enum Mode {
  kOne,     // a warp a segment
  kLine,    // equal stretches of the line of all segments, joined by a second kernel
  kCluster  // a cluster of CTAs a segment, joined through distributed shared memory
};
constexpr int kMaxCluster = 8;      // portable
// A cluster a segment saves a launch and the workspace; it pays while a warp has
// no more than four steps (two where its CTAs would leave most SMs idle), and
// only while all clusters find room at once (16 clusters of 8 did not: 19 us where
// the line takes 10).  8 kv heads, 16 bits, device time against the line's: one
// request of 1009 tokens 6.0 us, 8.5; 4096 10.5, 11.4; 8192 15.4, 14.0; four
// requests of 2048 10.5, 12.9.  One kv head, 2048 tokens: 8.3, 7.1 (a launch less on
// the host); 4096: 11.3, 7.7.
constexpr int kClusterSteps = 4, kClusterStepsFew = 2, kClusterFew = 32;
constexpr int kClusterCtas = 128, kCluster8Ctas = 64;
// What beginning a segment costs, in steps: the line counts each segment as that
// much longer, so that a warp with many short ones gets fewer steps (64 ragged
// requests 8+8: 102 us with 1, 97 with 2, 97 with 3).
constexpr int kSegmentCost = 2;

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
  int num_pages, page_size, max_pages;
  int B, H, Hk, G, n_q, rows, groups;  // rows = G * n_q in `groups` groups of 8 NT
  int max_len, causal, workers, step_tokens, cluster;
  float scale_log2;
  float up;                      // 2^kUp: how many times too small the O of unfinished pieces is
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

__device__ __forceinline__ uint32_t bytes(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}

// Four int8 codes as four fp16 numbers: code + 128 (0 .. 255) taken as fp16 bits
// is a subnormal, (code + 128) 2^-24 exactly, which the MMA multiplies as any
// other number; three instructions where a conversion takes five (and eight to
// bf16).
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = bytes(u, 0, 0x4140);
  hi = bytes(u, 0, 0x4342);
}

// Four E4M3 codes of token t (word a) and of token t' (word b), as four pairs
// (t, t') of fp16 numbers, exactly.
__device__ __forceinline__ void e4m3_pairs(uint32_t a, uint32_t b, uint32_t* out) {
  const uint32_t x = bytes(a, b, 0x5140), y = bytes(a, b, 0x7362);
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(out[0]), "=r"(out[1])
      : "r"(x));
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(out[2]), "=r"(out[3])
      : "r"(y));
}

// two fp16 numbers / kApart
__device__ __forceinline__ uint32_t over_apart(uint32_t a) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x10001000u));
  return r;
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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// maximum over the lanes that hold the same two rows of S^T (other tokens)
__device__ __forceinline__ float token_max(float v) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Bulk copy of n bytes (a multiple of 16; both addresses 16-byte aligned),
// counted by `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t n, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(n), "r"(smem_u32(bar))
               : "memory");
}

// -------------------------------------------------------- shapes of a step
// Tokens of a step, about 8 KB of K and V.
constexpr int step_tokens(int d, int format) {
  return d == 128 ? (format == SAGE_KV_8P8 ? 32 : 16) : (format == SAGE_KV_8P8 ? 64 : 32);
}

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
  static constexpr int TOK = step_tokens(D, FMT);
  static constexpr int SUB = TOK / 16;                   // 16-token tiles of a step
  // a stage of the ring: K rows, V rows, K scales, V scales
  static constexpr int V_AT = TOK * KROW;
  static constexpr int KS_AT = V_AT + TOK * VROW;
  static constexpr int VS_AT = KS_AT + (KS ? TOK * 4 : 0);
  static constexpr int STAGE = VS_AT + (VS ? TOK * 4 : 0);
  static constexpr int TOKEN = KROW + VROW + (KS ? 4 : 0) + (VS ? 4 : 0);  // bytes of a token
};

inline __host__ __device__ int steps_of(int len, int tok) { return (len + tok - 1) / tok; }
// places of a segment in the line
inline __host__ __device__ int places_of(int len, int tok) { return len > 0 ? steps_of(len, tok) + kSegmentCost : 0; }
// places of a worker: at least total / workers (fp32 rounded up, since a 64-bit
// division is slow), the same number wherever it is asked for
__device__ __forceinline__ int64_t per_worker(int64_t total, int workers) {
  const int64_t per = static_cast<int64_t>(ceilf(__fdiv_ru(__ll2float_ru(total), static_cast<float>(workers))));
  return per > kMinSteps ? per : kMinSteps;
}

// steps of a warp of a cluster
__device__ __forceinline__ int cluster_steps(int steps, int cluster) {
  return (steps + cluster * kWarps - 1) / (cluster * kWarps);
}

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
// A worker's part of the line: where it begins, and how many of its places are
// left, counted from the first that holds a step.  A segment takes kSegmentCost
// places without a step, then one for each of its steps.
struct Stretch {
  Cursor cur;
  int64_t left;
};

// The prefix sums of a CTA: places before each request, and how far into its
// last step each one reaches (its length follows from the two).
struct Requests {
  const int* places;    // [B + 1]
  const uint8_t* last;  // [B]
};

// Warp-major numbers: few workers then stand on as many SMs as they can.
__device__ __forceinline__ int worker_of(int warp) { return warp * gridDim.x + blockIdx.x; }

template <typename S, Mode MODE>
__device__ __forceinline__ Stretch stretch_of(const DecodeParams& p, const Requests& q, int warp) {
  Stretch w;
  const int HZ = p.Hk * p.groups;
  w.left = 0;
  w.cur.b = -1;
  if (MODE == kLine) {
    const int worker = worker_of(warp);
    const int64_t total = static_cast<int64_t>(q.places[p.B]) * HZ;
    const int64_t per = per_worker(total, p.workers);
    const int64_t at = worker * per;
    const int64_t end = worker < p.workers ? min(total, at + per) : 0;
    if (at >= end) return w;
    // the request that holds place `at`: the last one with places * HZ <= at
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<int64_t>(q.places[mid]) * HZ <= at) lo = mid; else hi = mid;
    }
    const int places = q.places[lo + 1] - q.places[lo];
    int64_t in = at - static_cast<int64_t>(q.places[lo]) * HZ;
    // in / places by fp32 (a 64-bit division is slow), then put right: it is off by
    // one at most for any head count below 2^22
    int z = min(static_cast<int>(__ll2float_rn(in) / static_cast<float>(places)), HZ - 1);
    in -= static_cast<int64_t>(z) * places;
    for (; in < 0; in += places) --z;
    for (; in >= places; in -= places) ++z;
    const int place = static_cast<int>(in);
    w.cur.b = lo;
    w.cur.z = z;
    w.cur.steps = places - kSegmentCost;
    w.cur.step = max(0, place - kSegmentCost);
    w.cur.len = (w.cur.steps - 1) * S::TOK + 1 + q.last[lo];
    // places at the segment's beginning that hold no step
    w.left = end - at - max(0, kSegmentCost - place);
  } else {
    const int segment = MODE == kOne ? worker_of(warp) : blockIdx.x / p.cluster;
    if (segment >= p.B * HZ) return w;
    w.cur.b = segment / HZ;
    w.cur.z = segment - w.cur.b * HZ;
    w.cur.step = 0;
    w.cur.len = clamp_len(p, p.lens[w.cur.b]);
    w.cur.steps = steps_of(w.cur.len, S::TOK);
    w.left = w.cur.steps;
    if (MODE == kCluster) {  // its warps take equal stretches, first those of the first warps
      const int per = cluster_steps(w.cur.steps, p.cluster);
      w.cur.step = (warp * p.cluster + blockIdx.x % p.cluster) * per;
      w.left = max(0, min(per, w.cur.steps - w.cur.step));
    }
  }
  return w;
}

// On to the next segment that has steps (the caller knows that places are left
// beyond this one); those it has without a step are taken off `left`.
template <typename S>
__device__ __forceinline__ void next_segment(const DecodeParams& p, const Requests& q, Cursor& c, int64_t& left) {
  left -= kSegmentCost;
  c.step = 0;
  if (++c.z < p.Hk * p.groups) return;
  c.z = 0;
  if (left <= 0) return;
  do {
    ++c.b;
    c.steps = q.places[c.b + 1] - q.places[c.b] - kSegmentCost;
  } while (c.steps <= 0);
  c.len = (c.steps - 1) * S::TOK + 1 + q.last[c.b];
}

// A loading warp: each of its lanes feeds the ring of one consuming warp, so that
// one instruction stream serves several.  The page numbers of a lane's next step
// are read while the current one is copied.
template <typename S, Mode MODE>
__device__ __forceinline__ void feed(const DecodeParams& p, const Requests& q, uint8_t* smem, uint64_t* full,
                                     uint64_t* empty, uint32_t* absent, volatile int* abort_flag, int feeder,
                                     int lane) {
  Stretch w;
  w.left = 0;
  // A bulk copy takes its warp about 120 cycles, whichever lane it is for, and a
  // step has to be begun every 350 cycles of an SM to keep HBM busy: with two
  // copies a step one warp does for all (and in a fairer order: 90 us where four
  // take 95, 131072 tokens of 16 bits), with more all four share them (97 us
  // where one takes 125, 64 requests of 8+8).
  const bool one_page = p.page_size % S::TOK == 0;  // a step lies in one page
  const int feeders = (one_page ? 1 : S::SUB) * (2 + S::KS + S::VS) <= 2 ? 1 : kFeeders;
  const int of = feeder < feeders ? feeder + lane * feeders : kWarps;  // the warp that this lane feeds
  if (of < kWarps) w = stretch_of<S, MODE>(p, q, of);
  int64_t left = w.left;
  int issued = 0;  // stages filled, kStages at most
  uint8_t* const ring = smem + of * (kStages * S::STAGE);
  full += of * kStages;
  empty += of * kStages;
  absent += of * kStages;
  Cursor& c = w.cur;
  int tile_page = 0, tile_off = 0;                  // page index and offset of the next step
  int ids[S::SUB];                                  // its pages, one a tile (or one)
  auto fetch = [&]() {
#pragma unroll
    for (int s = 0; s < S::SUB; ++s) {
      if (s > 0 && one_page) break;
      int pg = tile_page, off = tile_off + 16 * s;
      while (off >= p.page_size) {
        off -= p.page_size;
        ++pg;
      }
      const bool in = c.step * S::TOK + 16 * s < c.len;
      ids[s] = in ? p.table[static_cast<int64_t>(c.b) * p.max_pages + pg] : -1;
    }
  };
  auto seek = [&]() {
    const int t = c.step * S::TOK;
    tile_page = t / p.page_size;
    tile_off = t - tile_page * p.page_size;
  };
  if (left > 0) {
    seek();
    fetch();
  }
  int slot = 0;
  uint32_t parity = 0, round = 0;
  uint64_t since = 0;
  while (__any_sync(0xffffffffu, left > 0)) {
    bool moved = false;
    if (left > 0 && (round == 0 || mbar_test_wait(empty + slot, parity ^ 1))) {
      moved = true;
      const int64_t head = static_cast<int64_t>(c.z / p.groups) * p.page_size;
      const uint32_t dst = smem_u32(ring + slot * S::STAGE);
      uint64_t* const bar = full + slot;
      uint32_t gone = 0, bytes = 0;
      const int tiles = one_page ? 1 : S::SUB;
      const int n = one_page ? S::TOK : 16;
#pragma unroll
      for (int s = 0; s < S::SUB; ++s) {
        if (s >= tiles) break;
        if (static_cast<uint32_t>(ids[s]) < static_cast<uint32_t>(p.num_pages)) bytes += n * S::TOKEN;
        else gone |= (one_page ? (1u << S::SUB) - 1 : 1u << s);
      }
      absent[slot] = gone;
      mbar_arrive_expect_tx(bar, bytes);
      int off = tile_off;
#pragma unroll
      for (int s = 0; s < S::SUB; ++s) {
        if (s >= tiles) break;
        const int64_t page = ids[s], row = head + off;
        if (static_cast<uint32_t>(ids[s]) < static_cast<uint32_t>(p.num_pages)) {
          const int at = 16 * s;
          bulk_load(dst + at * S::KROW, p.k + page * p.k_page + row * S::KROW, n * S::KROW, bar);
          bulk_load(dst + S::V_AT + at * S::VROW, p.v + page * p.v_page + row * S::VROW, n * S::VROW, bar);
          if (S::KS) bulk_load(dst + S::KS_AT + at * 4, p.ks + page * p.ks_page + row, n * 4, bar);
          if (S::VS) bulk_load(dst + S::VS_AT + at * 4, p.vs + page * p.vs_page + row, n * 4, bar);
        }
        off += 16;
        if (off >= p.page_size) off = 0;
      }
      --left;
      if (issued < kStages) ++issued;
      if (left > 0) {
        tile_off += S::TOK;
        while (tile_off >= p.page_size) {
          tile_off -= p.page_size;
          ++tile_page;
        }
        if (++c.step == c.steps) {
          next_segment<S>(p, q, c, left);
          seek();
        }
        if (left > 0) fetch();
      }
      if (++slot == kStages) {
        slot = 0;
        ++round;
        parity ^= 1;
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
      since = 0;
    } else {  // every ring is full: nothing to do for a while
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
      const uint64_t now = globaltimer();
      if (since == 0) since = now;
      if (__any_sync(0xffffffffu, now - since > p.timeout_ns)) {
        if (lane == 0) atomicOr(&g_error_word, ERR_TIMEOUT | (0xD1u << 8));
        *abort_flag = 1;
        break;
      }
      __nanosleep(20);
    }
  }
  // The copies under way write to this CTA's memory: stay until they have landed,
  // also where a consumer has given up (as long again at most, and 10 ms at least).
  since = globaltimer();
  const uint64_t limit = p.timeout_ns > 10000000 ? p.timeout_ns : 10000000;
  while (issued-- > 0) {
    if (--slot < 0) {
      slot = kStages - 1;
      parity ^= 1;
    }
    while (!mbar_test_wait(full + slot, parity) && globaltimer() - since < limit) __nanosleep(100);
  }
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the address of this CTA's shared address `a` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}

// pieces of four channels of a row, joined: o (in units of 2^m) and l
struct Four {
  float o[4], m, l;
};
// `n` pieces, piece i's (m, l) and O at the addresses that `ml` and `o` give
template <typename ML, typename O>
__device__ __forceinline__ Four join_four(int n, ML ml, O o) {
  Four r = {{0.f, 0.f, 0.f, 0.f}, -INFINITY, 0.f};
  float2 w[kWarps];
  float4 x[kWarps];
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    w[i] = make_float2(-INFINITY, 0.f);
    if (i < n) {
      w[i] = *ml(i);
      x[i] = *o(i);
    }
    r.m = fmaxf(r.m, w[i].x);
  }
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < n && w[i].x != -INFINITY) {
      const float f = exp2_fast(w[i].x - r.m);
      r.l += w[i].y * f;
      r.o[0] += x[i].x * f;
      r.o[1] += x[i].y * f;
      r.o[2] += x[i].z * f;
      r.o[3] += x[i].w * f;
    }
  }
  return r;
}

// Bytes of a cluster CTA's inbox: (m, l) and O of four channels of every row.
template <int D, int ROWS>
constexpr int inbox_bytes() {
  return ROWS * (D / 4) * 24;
}

// Joins the pieces that the consuming warps of a cluster have left in their rings
// (O [ROWS][D] and (m, l) [ROWS] each).  Each CTA joins its own eight, then sends
// every unit of four channels to the CTA that writes it (remote stores: nobody
// waits for them but the barrier), which joins what the CTAs sent.  Reading the 64
// pieces of a cluster remotely took 3 us where this takes 1.
template <typename T, int D, int ROWS>
__device__ __forceinline__ void join_cluster(const DecodeParams& p, int b, int h, int row0, uint8_t* smem,
                                             int ring_bytes) {
  static_assert(kMaxCluster <= kWarps, "join_four takes kWarps pieces");
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
  const int rows = min(ROWS, p.rows - row0);
  const int units = rows * (D / 4);
  const int rank = blockIdx.x % p.cluster;
  // the inbox behind the rings: float4 [unit / cluster][source], then float2 alike
  uint8_t* const box = smem + kWarps * ring_bytes;
  const int places = (units + p.cluster - 1) / p.cluster * p.cluster;
  cluster_wait();  // of the kernel's beginning: every CTA is there
  for (int u = threadIdx.x; u < units; u += kWarps * 32) {
    const int r = u / (D / 4), ch = (u - r * (D / 4)) * 4;
    const Four f = join_four(
        kWarps,
        [&](int i) { return reinterpret_cast<const float2*>(smem + i * ring_bytes + ROWS * D * 4) + r; },
        [&](int i) { return reinterpret_cast<const float4*>(smem + i * ring_bytes + (r * D + ch) * 4); });
    const int place = u / p.cluster, to = u - place * p.cluster;
    const uint32_t a = cluster_addr(smem_u32(box) + (place * p.cluster + rank) * 16, to);
    const uint32_t c = cluster_addr(smem_u32(box) + places * 16 + (place * p.cluster + rank) * 8, to);
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(f.o[0]), "f"(f.o[1]), "f"(f.o[2]),
                 "f"(f.o[3])
                 : "memory");
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(c), "f"(f.m), "f"(f.l) : "memory");
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  for (int place = threadIdx.x; place * p.cluster + rank < units; place += kWarps * 32) {
    const int u = place * p.cluster + rank;
    const int r = u / (D / 4), ch = (u - r * (D / 4)) * 4;
    const Four f = join_four(
        p.cluster,
        [&](int i) { return reinterpret_cast<const float2*>(box + places * 16) + place * p.cluster + i; },
        [&](int i) { return reinterpret_cast<const float4*>(box) + place * p.cluster + i; });
    const int row = row0 + r, qi = row / p.G;
    const int64_t out = (static_cast<int64_t>(b) * p.H + h * p.G + (row - qi * p.G)) * p.n_q + qi;
    const float g = f.l > 0.f ? p.up / f.l : 0.f;
    *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.o) + out * D + ch) =
        make_uint2(pack16<T>(f.o[0] * g, f.o[1] * g), pack16<T>(f.o[2] * g, f.o[3] * g));
    if (p.lse != nullptr && ch == 0)
      p.lse[out] = f.l > 0.f ? (f.m + log2f(f.l)) * 0.69314718055994531f : -INFINITY;
  }
}

template <typename T, int D, int FMT, int NT, Mode MODE>
__global__ void __launch_bounds__((kWarps + kFeeders) * 32, 1) k_attn_decode(const DecodeParams p) {
  using S = Step<D, FMT>;
  // int8 K and E4M3 V become fp16 whatever the model's type is
  using TK = typename std::conditional<FMT == SAGE_KV_16, T, __half>::type;
  using TV = typename std::conditional<FMT == SAGE_KV_8P8, __half, T>::type;
  constexpr bool kScaledQ = !std::is_same<T, TK>::value;
  constexpr bool kHalfP = std::is_same<TV, __half>::value;
  constexpr float kUp = lift_of(kHalfP, FMT);
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[kWarps * kStages], s_empty[kWarps * kStages];
  __shared__ uint32_t s_absent[kWarps * kStages];  // tiles of a stage that are on no page
  __shared__ int s_scan[kWarps + kFeeders];
  __shared__ int s_abort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  int* s_places = reinterpret_cast<int*>(smem + kWarps * kStages * S::STAGE);  // kLine only
  uint8_t* s_last = reinterpret_cast<uint8_t*>(s_places + p.B + 1);
  const Requests q = {s_places, s_last};

  if (threadIdx.x < kWarps * kStages) {
    mbar_init(s_full + threadIdx.x, 1);
    mbar_init(s_empty + threadIdx.x, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) s_abort = 0;
  after_previous();  // and before the join may be placed: it reads the lengths while this grid runs
  if (MODE == kCluster) {  // before the first remote store, all CTAs have started
    __syncwarp();
    cluster_arrive();
  }
  if (MODE == kLine) {
    // the join's CTAs may be placed now; they wait for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int run = 0;
    for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
      const int b = b0 + threadIdx.x;
      const int len = b < p.B ? clamp_len(p, p.lens[b]) : 0;
      int v = places_of(len, S::TOK);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = v;
      __syncthreads();
      int before = run;
      for (int w = 0; w < kWarps + kFeeders; ++w) {
        if (w < warp) before += s_scan[w];
        run += s_scan[w];
      }
      if (b < p.B) {
        s_places[b + 1] = before + v;
        s_last[b] = static_cast<uint8_t>((len - 1) % S::TOK);
      }
    }
    if (threadIdx.x == 0) s_places[0] = 0;
  }
  __syncthreads();
  // Two tiles of rows need more registers than 12 warps get at launch: the four
  // loading warps give theirs up (56 + 2 * 224 = 3 * 168).
  constexpr bool kShift = NT > 1;
  if (warp >= kWarps) {
    if (kShift) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    feed<S, MODE>(p, q, smem, s_full, s_empty, s_absent, &s_abort, warp - kWarps, lane);
    return;
  }

  if (kShift) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
  Stretch st = stretch_of<S, MODE>(p, q, warp);
  if (MODE == kLine ? st.left <= 0 : st.cur.b < 0) return;
  Cursor& cur = st.cur;
  int64_t left = st.left;
  uint8_t* const ring = smem + warp * (kStages * S::STAGE);
  uint64_t* const full = s_full + warp * kStages;
  uint64_t* const empty = s_empty + warp * kStages;
  int slot = 0;
  uint32_t parity = 0;
  bool first_piece = true;
  while (true) {
    // one piece: steps [cur.step, stop) of one segment
    const int stop = static_cast<int>(min(static_cast<int64_t>(cur.steps), cur.step + left));
    const bool whole = MODE == kOne || (cur.step == 0 && stop == cur.steps);
    const int h = cur.z / p.groups, row0 = (cur.z - h * p.groups) * ROWS;

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
    float to_log2 = p.scale_log2;
    float base_s[NT][2];  // where a score's sum starts
    float back[NT][2];    // of bf16 q that became fp16: each row's power of two
#pragma unroll
    for (int n = 0; n < NT; ++n) base_s[n][0] = base_s[n][1] = 0.f;
    if (S::KB == 1) {
      if (kScaledQ) {
        // bf16 q to fp16, each row times the power of two that brings its largest to
        // [2^13, 2^14): exact down to 2^-28 of it, and what is lost below is less than
        // fp32 loses in the sum
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 f = unpack16<T>(qf[n][i][e]);
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));  // of row g
          const int ex = static_cast<int>(__float_as_uint(top) >> 23 & 255);
          const int k = top > 0.f ? min(127, 13 - (ex - 127)) : 0;  // >= -115
          const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
          const float down = __uint_as_float(static_cast<uint32_t>(127 + 12 - k) << 23);  // 2^(12 - k)
          back[n][0] = __shfl_sync(0xffffffffu, down, 8 * c);
          back[n][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 f = unpack16<T>(qf[n][i][e]);
              qf[n][i][e] = pack16<__half>(f.x * up, f.y * up);
            }
        }
      }
      // code + 128, as the bits of an fp16 number, is (code + 128) 2^-24: the sums
      // start at -128 2^-24 sum q, and end 2^24 times too small
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = unpack16<__half>(qf[n][i][e]);
            sum += f.x + f.y;
          }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);  // of row g
        sum *= -128.f / 16777216.f;
        base_s[n][0] = __shfl_sync(0xffffffffu, sum, 8 * c);
        base_s[n][1] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
      }
      to_log2 *= kScaledQ ? 4096.f : 16777216.f;  // half of the 2^24 is in `back`: neither leaves fp32
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

    // m: kUp below the largest score, or below one less by kSlack at most; l: sum of
    // 2^(s - m).  O is summed in units of `unit`, the largest delta_V so far up to a
    // factor of kUnitSlack, so that P delta_V / unit fits fp16 whatever V's range.
    float acc[NT][D / 16][4];
    float m[NT][2], l[NT][2];
    float unit = S::VS ? kTinyScale : 1.f, per_unit = S::VS ? 1.f / kTinyScale : 1.f;
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
      uint8_t* const base = ring + slot * S::STAGE;
      const bool there = mbar_wait(full + slot, parity, &s_abort, p.timeout_ns, 0xD0);
      if (!__all_sync(0xffffffffu, there)) {  // given up: the error word says so
        if (MODE != kCluster) return;
        break;  // the other CTAs of the cluster will read this one's memory
      }
      const int t0 = cur.step * S::TOK;
      const uint32_t gone = s_absent[warp * kStages + slot];
      // Behind the last token the page may hold anything, and a tile on no page
      // was not copied.  Their scores are masked below; their V is zeroed here,
      // since 0 * NaN would reach the sums.
      if (t0 + S::TOK > cur.len || gone != 0) {
#pragma unroll
        for (int u = 0; u < S::SUB; ++u) {
          const int have = gone >> u & 1 ? 0 : min(16, max(0, cur.len - t0 - 16 * u));
          for (int i = have * S::VROW + 16 * lane; i < 16 * S::VROW; i += 512)
            *reinterpret_cast<uint4*>(base + S::V_AT + 16 * u * S::VROW + i) = make_uint4(0, 0, 0, 0);
          if (S::VS && lane >= have && lane < 16)
            *reinterpret_cast<float*>(base + S::VS_AT + (16 * u + lane) * 4) = 0.f;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }

      // ---- sums of products with K
      float s[NT][S::SUB][4];
#pragma unroll
      for (int u = 0; u < S::SUB; ++u) {
        const uint8_t* const kb = base + (16 * u + g) * S::KROW + c * 16;
        float s2[NT][4];  // a second accumulator: two chains of products, half as long
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[n][u][e] = base_s[n][e & 1];
            s2[n][e] = 0.f;
          }
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
              for (int n = 0; n < NT; ++n)
                mma16816<TK>(y ? s2[n] : s[n][u], a, qf[n][2 * x + y][0], qf[n][2 * x + y][1]);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t a[4];
              codes_to_half(a0[y], a[0], a[2]);
              codes_to_half(a1[y], a[1], a[3]);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816<TK>(y & 1 ? s2[n] : s[n][u], a, qf[n][(4 * x + y) % (D / 16)][0],
                             qf[n][(4 * x + y) % (D / 16)][1]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][u][e] += s2[n][e];
      }
      // ---- V to registers; the stage is free once all of it is
      constexpr int VWORDS = S::VW / 4;
      uint32_t vr[S::SUB][4][S::VC][VWORDS];
      float ks[S::SUB][2], vs[S::SUB][2];
#pragma unroll
      for (int u = 0; u < S::SUB; ++u) {
        const uint8_t* const vb = base + S::V_AT + (16 * u + 2 * c) * S::VROW + g * S::VW;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int x = 0; x < S::VC; ++x) {
            const uint8_t* const v0 = vb + ((j & 1) + 8 * (j >> 1)) * S::VROW + x * 8 * S::VW;
            if (S::VW == 16) {
              const uint4 r = *reinterpret_cast<const uint4*>(v0);
              vr[u][j][x][0] = r.x;
              vr[u][j][x][1] = r.y;
              vr[u][j][x][2 % VWORDS] = r.z;
              vr[u][j][x][3 % VWORDS] = r.w;
            } else {
              const uint2 r = *reinterpret_cast<const uint2*>(v0);
              vr[u][j][x][0] = r.x;
              vr[u][j][x][1] = r.y;
            }
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ks[u][e] = S::KS ? *reinterpret_cast<const float*>(base + S::KS_AT + (16 * u + 8 * e + g) * 4) : 1.f;
          vs[u][e] = S::VS ? *reinterpret_cast<const float*>(base + S::VS_AT + (16 * u + 8 * e + g) * 4) : 1.f;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + slot);
      if (++slot == kStages) {
        slot = 0;
        parity ^= 1;
      }

      // ---- scores, in units of log2
#pragma unroll
      for (int u = 0; u < S::SUB; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = S::KS ? to_log2 * ks[u][e] : to_log2;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[n][u][2 * e] *= kScaledQ ? f * back[n][0] : f;
            s[n][u][2 * e + 1] *= kScaledQ ? f * back[n][1] : f;
          }
        }
      // ---- masks: the end of the cache, later query tokens' keys, no page
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
      // ---- running maxima: reduced over the lanes, and O rescaled, only where a
      // score has outgrown m by kSlack (in log2) or a delta_V the unit.  Directed
      // roundings keep P within fp16 where scores are so large that their steps are not
      // small beside kUp.
      bool grew = false;
      float top[NT][2], top_v = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[n][0][e], s[n][0][e + 2]);
#pragma unroll
          for (int u = 1; u < S::SUB; ++u) t = fmaxf(t, fmaxf(s[n][u][e], s[n][u][e + 2]));
          top[n][e] = t;
          grew |= t > __fadd_rd(m[n][e], kSlack + kUp);
        }
      if (S::VS) {
#pragma unroll
        for (int u = 0; u < S::SUB; ++u) top_v = fmaxf(top_v, fmaxf(vs[u][0], vs[u][1]));
        grew |= top_v > kUnitSlack * unit;
      }
      if (__any_sync(0xffffffffu, grew)) {
        float down = 1.f;
        if (S::VS) {
          top_v = fmaxf(token_max(top_v), unit);
          per_unit = __frcp_rn(top_v);
          down = unit * per_unit;
          unit = top_v;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float t = fmaxf(__fadd_ru(token_max(top[n][e]), -kUp), m[n][e]);
            alpha[e] = t == m[n][e] ? 1.f : exp2_fast(m[n][e] - t);
            m[n][e] = t;
            l[n][e] *= alpha[e];
            if (S::VS) alpha[e] *= down;
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
      uint32_t least = 0xffffffffu;  // the bits of the smallest P that counts, less kNothing
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m0[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0], m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
        for (int u = 0; u < S::SUB; ++u) {
          float* const e = s[n][u];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = exp2_fast(e[i] - m0[i & 1]);
          l[n][0] += e[0] + e[2];
          l[n][1] += e[1] + e[3];
          if (S::VS) {
            const float f[2] = {vs[u][0] * per_unit, vs[u][1] * per_unit};
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] *= f[i >> 1];
          }
          if (kHalfP) {
#pragma unroll
            for (int i = 0; i < 4; ++i) least = min(least, __float_as_uint(e[i]) - kNothing);
          }
        }
      }
      const bool small = kHalfP && __any_sync(0xffffffffu, least < kSmall - kNothing);
      const float rest = small ? kApart : 1.f;
      uint32_t pf[NT][S::SUB][2], pl[NT][S::SUB][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < S::SUB; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t hi = pack16<TV>(s[n][u][2 * i], s[n][u][2 * i + 1]);
            const float2 f = unpack16<TV>(hi);
            pf[n][u][i] = transpose8x8(hi);
            pl[n][u][i] = transpose8x8(pack16<TV>((s[n][u][2 * i] - f.x) * rest, (s[n][u][2 * i + 1] - f.y) * rest));
          }
      // `apart`: the second numbers are kApart times as large
      auto add_v = [&](auto apart) {
#pragma unroll
        for (int u = 0; u < S::SUB; ++u)
#pragma unroll
          for (int x = 0; x < S::VC; ++x)
#pragma unroll
            for (int i = 0; i < VWORDS; ++i) {
              const uint32_t w0 = vr[u][0][x][i], w1 = vr[u][1][x][i], w2 = vr[u][2][x][i], w3 = vr[u][3][x][i];
              if (S::VB == 2) {
                const int tile = (VWORDS * x + i) % (D / 16);
                const uint32_t a[4] = {bytes(w0, w1, 0x5410), bytes(w0, w1, 0x7632), bytes(w2, w3, 0x5410),
                                       bytes(w2, w3, 0x7632)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  mma16816<TV>(acc[n][tile], a, pf[n][u][0], pf[n][u][1]);
                  if (decltype(apart)::value) {  // sums of their own
                    float low[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816<TV>(low, a, pl[n][u][0], pl[n][u][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[n][tile][e] += low[e] * (1.f / kApart);
                  } else {
                    mma16816<TV>(acc[n][tile], a, pl[n][u][0], pl[n][u][1]);
                  }
                }
              } else {
                uint32_t x01[4], x23[4];
                e4m3_pairs(w0, w1, x01);
                e4m3_pairs(w2, w3, x23);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int tile = (2 * (VWORDS * x + i) + y) % (D / 16);
                  uint32_t a[4] = {x01[2 * y], x01[2 * y + 1], x23[2 * y], x23[2 * y + 1]};
#pragma unroll
                  for (int n = 0; n < NT; ++n) mma16816<TV>(acc[n][tile], a, pf[n][u][0], pf[n][u][1]);
                  if (decltype(apart)::value) {  // V / kApart, exactly: E4M3's numbers are multiples of 2^-9
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = over_apart(a[e]);
                  }
#pragma unroll
                  for (int n = 0; n < NT; ++n) mma16816<TV>(acc[n][tile], a, pl[n][u][0], pl[n][u][1]);
                }
              }
            }
      };
      if (kHalfP && small) add_v(std::integral_constant<bool, kHalfP>());
      else add_v(std::false_type());
    }

    // ---- end of the piece
    // Channels of a lane: VE neighbours of each of the VC pieces (a V piece's
    // channels are spread over VE / 2 tiles, two a tile).
    constexpr int TILES = S::VE / 2;
    // O of an unfinished piece goes without the lift, for which V near bf16's end
    // leaves no room
    const float in = unit * (1.f / (1 << lift_of(kHalfP, FMT)));
    // where an unfinished piece goes: the workspace, or the warp's own ring
    const int64_t slot_p = 2 * static_cast<int64_t>(worker_of(warp)) + (first_piece ? 0 : 1);
    float* const part_o = MODE == kCluster ? reinterpret_cast<float*>(ring) : p.part_o + slot_p * ROWS * D;
    float2* const part_ml =
        MODE == kCluster ? reinterpret_cast<float2*>(ring + ROWS * D * sizeof(float)) : p.part_ml + slot_p * ROWS;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int rg = 8 * n + 2 * c + e, r = row0 + rg;
        if (r >= p.rows) continue;
        if (MODE == kOne || (MODE == kLine && whole)) {
          const int qi = r / p.G, hh = h * p.G + (r - qi * p.G);
          const int64_t out = (static_cast<int64_t>(cur.b) * p.H + hh) * p.n_q + qi;
          const float f = sum > 0.f ? unit / sum : 0.f;
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
            p.lse[out] = sum > 0.f ? (m[n][e] + log2f(sum)) * 0.69314718055994531f : -INFINITY;
        } else {
          float* dst = part_o + rg * D + g * S::VE;
#pragma unroll
          for (int x = 0; x < S::VC; ++x)
#pragma unroll
            for (int i = 0; i < TILES; i += 2)
              *reinterpret_cast<float4*>(dst + x * 8 * S::VE + 2 * i) =
                  make_float4(acc[n][x * TILES + i][e] * in, acc[n][x * TILES + i][e + 2] * in,
                              acc[n][x * TILES + i + 1][e] * in, acc[n][x * TILES + i + 1][e + 2] * in);
          if (g == 0) part_ml[rg] = make_float2(m[n][e], sum);
        }
      }
    if (MODE == kCluster) {
      join_cluster<T, D, ROWS>(p, cur.b, h, row0, smem, kStages * S::STAGE);
      return;
    }
    first_piece = false;
    if (left <= 0) return;
    next_segment<S>(p, q, cur, left);
    if (left <= 0) return;
  }
}

// ------------------------------------------------------------------ join
// A CTA joins `per_cta` rows of one segment, all of which have the same n
// pieces.  kJoinLoads pieces of O are in flight while the weights exp2(m_i - m)
// are formed, and after that in each round.  Up to 32 pieces a warp joins
// a row by itself; with more (or one row a CTA, where rows are few) the warps
// share each row's pieces and are added in order.  Either way the order of the
// sum depends on the sizes alone.  Rows of requests without tokens are zeros.
constexpr int kJoinLoads = 12;
constexpr int kMaxPieces = kSms * kWarps;  // a segment has at most one of each worker

// kJoinLoads pieces of a row (a lane's D / 32 channels of each): i0, i0 + stride, ...
template <int D>
__device__ __forceinline__ void load_pieces(float (*x)[D / 32], const float* po, int64_t piece, int late, int i0,
                                            int stride, int n) {
  constexpr int PER = D / 32;
#pragma unroll
  for (int j = 0; j < kJoinLoads; ++j) {
    const int i = i0 + j * stride;
#pragma unroll
    for (int e = 0; e < PER; ++e) x[j][e] = 0.f;
    if (i < n) {
      const float* src = po + (2 * i + (i == 0 ? late : 0)) * piece;
      if (PER == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src);
        x[j][0] = f.x;
        x[j][1] = f.y;
        x[j][PER - 2] = f.z;
        x[j][PER - 1] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(src);
        x[j][0] = f.x;
        x[j][1] = f.y;
      }
    }
  }
}

template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) k_attn_join(const DecodeParams p, int rows_per_group, int per_cta,
                                                                int parts) {
  constexpr int PER = D / 32;
  __shared__ float s_w[kMaxPieces];
  __shared__ float s_o[WARPS][D];
  __shared__ float s_m[WARPS], s_l[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int HZ = p.Hk * p.groups;
  // grid: x = segment of the request and part of its rows, y = request
  const int z = blockIdx.x / parts, h = z / p.groups, row0 = (z - h * p.groups) * rows_per_group;
  const int b = blockIdx.y;
  const int first = (blockIdx.x - z * parts) * per_cta;
  const int last = min(min(first + per_cta, rows_per_group), p.rows - row0);
  if (first >= last) return;
  // where row rg of the segment goes
  auto out_of = [&](int rg) {
    const int r = row0 + rg, qi = r / p.G;
    return (static_cast<int64_t>(b) * p.H + h * p.G + (r - qi * p.G)) * p.n_q + qi;
  };
  // The lengths are inputs: the steps before this request and in all are
  // counted while the pieces are still being computed.
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < p.B; i += WARPS * 32) {
    const int v = places_of(clamp_len(p, p.lens[i]), p.step_tokens);
    all += v;
    if (i < b) before += v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  __shared__ int2 s_steps[WARPS];
  if (lane == 0) s_steps[warp] = make_int2(before, all);
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    before += s_steps[w].x;
    all += s_steps[w].y;
  }
  const int places = places_of(clamp_len(p, p.lens[b]), p.step_tokens);
  after_previous();
  if (places == 0) {
    for (int rg = first + warp; rg < last; rg += WARPS) {
      const int64_t out = out_of(rg);
      uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<T*>(p.o) + out * D);
      for (int i = lane; i < D / 2; i += 32) dst[i] = 0;
      if (p.lse != nullptr && lane == 0) p.lse[out] = -INFINITY;
    }
    return;
  }
  const int64_t total = static_cast<int64_t>(all) * HZ;
  const int64_t per = per_worker(total, p.workers);
  const int64_t s0 = static_cast<int64_t>(before) * HZ + static_cast<int64_t>(z) * places;
  const int w0 = static_cast<int>((s0 + kSegmentCost) / per), n = static_cast<int>((s0 + places - 1) / per) - w0 + 1;
  if (n == 1) return;  // one piece: finished where it was computed
  // a worker's first piece is in its first place, any other in its second
  const int late = w0 * per < s0 ? 1 : 0;
  const float2* ml = p.part_ml + static_cast<int64_t>(2 * w0) * rows_per_group;
  const float* po = p.part_o + static_cast<int64_t>(2 * w0) * rows_per_group * D + lane * PER;
  const int64_t piece = static_cast<int64_t>(rows_per_group) * D;

  if (n <= (per_cta > 1 ? 32 : kJoinLoads)) {
    for (int rg = first + warp; rg < last; rg += WARPS) {
      const float2 own = lane < n ? ml[(2 * lane + (lane == 0 ? late : 0)) * rows_per_group + rg]
                                  : make_float2(-INFINITY, 0.f);
      const float* row = po + static_cast<int64_t>(rg) * D;
      float x[kJoinLoads][PER], o[PER];
      load_pieces<D>(x, row, piece, late, 0, 1, n);
      const float m = warp_max(own.x);
      const float w = own.x == -INFINITY ? 0.f : exp2_fast(own.x - m);
      const float l = warp_sum(own.y * w);
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] = 0.f;
      for (int i0 = 0;;) {
#pragma unroll
        for (int j = 0; j < kJoinLoads; ++j) {
          const float f = __shfl_sync(0xffffffffu, w, (i0 + j) & 31);
#pragma unroll
          for (int e = 0; e < PER; ++e) o[e] += f * x[j][e];
        }
        i0 += kJoinLoads;
        if (i0 >= n) break;
        load_pieces<D>(x, row, piece, late, i0, 1, n);
      }
      const float f = l > 0.f ? p.up / l : 0.f;
      const int64_t out = out_of(rg);
      uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<T*>(p.o) + out * D + lane * PER);
#pragma unroll
      for (int e = 0; e < PER / 2; ++e) dst[e] = pack16<T>(o[2 * e] * f, o[2 * e + 1] * f);
      if (p.lse != nullptr && lane == 0)
        p.lse[out] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    return;
  }

  for (int rg = first; rg < last; ++rg) {
    constexpr int kOwn = (kMaxPieces + WARPS * 32 - 1) / (WARPS * 32);
    float2 own[kOwn];
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const int i = threadIdx.x + j * WARPS * 32;
      own[j] = i < n ? ml[(2 * i + (i == 0 ? late : 0)) * rows_per_group + rg] : make_float2(-INFINITY, 0.f);
      m = fmaxf(m, own[j].x);
    }
    const float* row = po + static_cast<int64_t>(rg) * D;
    float x[kJoinLoads][PER];
    load_pieces<D>(x, row, piece, late, warp, WARPS, n);
    m = warp_max(m);
    if (lane == 0) s_m[warp] = m;
    __syncthreads();
    m = warp_max(s_m[lane % WARPS]);
    float l = 0.f;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const int i = threadIdx.x + j * WARPS * 32;
      if (i < n) {
        const float w = own[j].x == -INFINITY ? 0.f : exp2_fast(own[j].x - m);
        l += own[j].y * w;
        s_w[i] = w;
      }
    }
    l = warp_sum(l);
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    float o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
    for (int i0 = warp;;) {
#pragma unroll
      for (int j = 0; j < kJoinLoads; ++j) {
        const int i = i0 + j * WARPS;
        const float f = i < n ? s_w[i] : 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] += f * x[j][e];
      }
      i0 += WARPS * kJoinLoads;
      if (i0 >= n) break;
      load_pieces<D>(x, row, piece, late, i0, WARPS, n);
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) s_o[warp][lane * PER + e] = o[e];
    __syncthreads();
    if (threadIdx.x < D / 2) {
      float ll = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        ll += s_l[w];
        a0 += s_o[w][2 * threadIdx.x];
        a1 += s_o[w][2 * threadIdx.x + 1];
      }
      const float f = ll > 0.f ? p.up / ll : 0.f;
      const int64_t out = out_of(rg);
      reinterpret_cast<uint32_t*>(reinterpret_cast<T*>(p.o) + out * D)[threadIdx.x] = pack16<T>(a0 * f, a1 * f);
      if (p.lse != nullptr && threadIdx.x == 0)
        p.lse[out] = ll > 0.f ? (m + log2f(ll)) * 0.69314718055994531f : -INFINITY;
    }
    // s_o and s_l are read above; the next row writes them after two barriers,
    // s_m and s_w after its first or before it, when every thread is past here
    __syncthreads();
  }
}

// ---------------------------------------------------------------- the plan
// Everything the host decides, from sizes alone (the lengths are on the
// device): how many query rows a warp takes, whether segments are split, and
// how many workers share the line.
struct Plan {
  int nt, groups, step_tokens, workers, ctas, cluster;
  Mode mode;
  size_t off_ml, bytes;
};

Plan plan_of(int B, int H, int H_kv, int n_q, int d, int max_len, int format) {
  Plan P = {};
  const int rows = H / H_kv * n_q;
  P.nt = rows <= 8 ? 1 : 2;
  P.groups = (rows + 8 * P.nt - 1) / (8 * P.nt);
  P.step_tokens = step_tokens(d, format);
  const int64_t steps = steps_of(max_len, P.step_tokens);
  const int64_t segments = static_cast<int64_t>(B) * H_kv * P.groups;
  int cluster = kMaxCluster;
  while (cluster > 1 && segments * cluster > (cluster == 8 ? kCluster8Ctas : kClusterCtas)) cluster /= 2;
  if (steps <= 4) {
    P.mode = kOne;
    P.workers = static_cast<int>(segments);
    P.ctas = static_cast<int>(std::max<int64_t>(std::min<int64_t>(kSms, segments), (segments + kWarps - 1) / kWarps));
  } else if (cluster > 1 && steps <= (segments * cluster < kClusterFew ? kClusterStepsFew : kClusterSteps) *
                                         static_cast<int64_t>(cluster) * kWarps) {
    P.mode = kCluster;
    P.cluster = cluster;
    P.ctas = static_cast<int>(segments) * cluster;
  } else {
    P.mode = kLine;
    const int64_t most = static_cast<int64_t>(kSms) * kWarps;
    const int64_t workers = std::min(most, (segments * (steps + kSegmentCost) + kMinSteps - 1) / kMinSteps);
    P.workers = static_cast<int>(workers);
    P.ctas = static_cast<int>(std::min<int64_t>(kSms, workers));
    const size_t slots = 2 * static_cast<size_t>(workers) * 8 * P.nt;
    P.off_ml = slots * d * sizeof(float);
    P.bytes = (P.off_ml + slots * sizeof(float2) + 255) / 256 * 256;
  }
  return P;
}

template <typename T, int D, int FMT, int NT, Mode MODE>
cudaError_t launch_one(const DecodeParams& p, const Plan& P, cudaStream_t st) {
  using S = Step<D, FMT>;
  constexpr int kRing = kWarps * kStages * S::STAGE;
  constexpr int kInbox = MODE == kCluster ? inbox_bytes<D, 8 * NT>() : 0;
  const size_t smem = kRing + kInbox + (MODE == kLine ? (static_cast<size_t>(p.B) + 1) * sizeof(int) + p.B : 0);
  auto* f = k_attn_decode<T, D, FMT, NT, MODE>;
  static OncePerDevice once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(
        f, cudaFuncAttributeMaxDynamicSharedMemorySize,
        kRing + kInbox + (MODE == kLine ? (kMaxBatch + 1) * static_cast<int>(sizeof(int)) + kMaxBatch : 0));
  });
  if (e != cudaSuccess) return e;
  if (MODE == kCluster) return launch_after(f, dim3(P.ctas), (kWarps + kFeeders) * 32, smem, st, P.cluster, p);
  e = launch_after(f, dim3(P.ctas), (kWarps + kFeeders) * 32, smem, st, 1, p);
  if (e != cudaSuccess || MODE != kLine) return e;
  // A CTA takes all rows of a segment (with a CTA a row, 2048 rows of two to five
  // pieces took 9 us where this takes 4), and fewer where that leaves SMs idle.
  const int in_group = std::min(8 * NT, p.rows);
  const int64_t segments = static_cast<int64_t>(p.groups) * p.Hk * p.B;
  int per_cta = in_group;
  while (per_cta > 1 && segments * ((in_group + per_cta - 1) / per_cta) < 2 * kSms) per_cta = (per_cta + 1) / 2;
  const int parts = (in_group + per_cta - 1) / per_cta;
  const dim3 join_grid(parts * p.groups * p.Hk, p.B);
  // a warp a row, or eight on one row
  if (per_cta > 1 && per_cta <= 4)
    return launch_after(k_attn_join<T, D, 4>, join_grid, 4 * 32, 0, st, 1, p, 8 * NT, per_cta, parts);
  return launch_after(k_attn_join<T, D, 8>, join_grid, 8 * 32, 0, st, 1, p, 8 * NT, per_cta, parts);
}
template <typename T, int D, int FMT, int NT>
cudaError_t launch_nt(const DecodeParams& p, const Plan& P, cudaStream_t st) {
  if (P.mode == kOne) return launch_one<T, D, FMT, NT, kOne>(p, P, st);
  if (P.mode == kCluster) return launch_one<T, D, FMT, NT, kCluster>(p, P, st);
  return launch_one<T, D, FMT, NT, kLine>(p, P, st);
}
template <typename T, int D, int FMT>
cudaError_t launch_fmt(const DecodeParams& p, const Plan& P, cudaStream_t st) {
  return P.nt == 1 ? launch_nt<T, D, FMT, 1>(p, P, st) : launch_nt<T, D, FMT, 2>(p, P, st);
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
  if (P.mode == kLine) {
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    p.part_o = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + P.off_ml);
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
  p.step_tokens = P.step_tokens;
  p.cluster = P.cluster;
  p.timeout_ns = a.timeout_ns;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.up = static_cast<float>(1 << lift_of(c.dtype == SAGE_F16 || c.format == SAGE_KV_8P8, c.format));
  if (c.dtype == SAGE_F16)
    return c.d == 64 ? launch_d<__half, 64>(p, P, c.format, st) : launch_d<__half, 128>(p, P, c.format, st);
  return c.d == 64 ? launch_d<__nv_bfloat16, 64>(p, P, c.format, st)
                   : launch_d<__nv_bfloat16, 128>(p, P, c.format, st);
}

}  // namespace sage
