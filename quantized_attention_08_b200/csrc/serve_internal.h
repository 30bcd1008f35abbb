// serve_internal.h -- declarations of the serving kernels (paged cache,
// rotary positions, decode attention) shared with the C entry points.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "sage.h"

namespace sage {

// Runs a set-up call (one that may be repeated, with the same effect) on each
// device's first use; a device whose call failed tries again.
class OncePerDevice {
 public:
  template <typename F>
  cudaError_t run(F f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return f();
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    if ((e = f()) == cudaSuccess) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<bool> done_[64] = {};
};

constexpr int kSms = 148;
// the smallest scale that a cache holds beside 0 (2^-100)
constexpr float kTinyScale = 7.88860905e-31f;

#if defined(__CUDACC__)
// A launch that may be placed while the kernel before it in the stream ends: the
// kernel begins with after_previous(), which waits for that one's end and for
// its writes.  Every block with work passes it, so that a kernel's end implies
// the end of all before it.  (A step is a chain of kernels of a few microseconds: their
// launches hide about a microsecond each in the ends of the ones before.)
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: CTAs of a thread-block cluster, 1 for none.
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
                         Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
#endif

struct SlotArgs {
  const int32_t* ctx_lens;
  const int32_t* new_lens;
  const int32_t* free_pages;
  const int32_t* free_used;  // may alias free_used_out
  int32_t* block_table;
  int32_t* seq_lens;         // may alias ctx_lens
  int32_t* cu_seqlens;
  int32_t* slot_map;
  int32_t* positions;
  int32_t* seq_ids;
  int32_t* free_used_out;
  int B, num_free, max_pages, page_size, T;
};
cudaError_t launch_kv_slots(const SlotArgs& a, cudaStream_t st);

constexpr int kMaxAxes = 4;

struct RopeArgs {
  const void* in[2];      // q, k (k may be nullptr)
  void* out[2];
  int64_t in_s[2][3];     // strides of batch, head, token (elements)
  int64_t out_s[2][3];
  int heads[2];
  const int32_t* pos;     // pos[a * pos_s[0] + b * pos_s[1] + n]
  int64_t pos_s[2];
  const float* inv_freq;  // [pairs]
  int sec_end[kMaxAxes];  // pair i belongs to the first axis a with i < sec_end[a]
  int axes, pairs;
  int B, N, d;
  int interleaved, bf16;
};
cudaError_t launch_rope_axes(const RopeArgs& a, cudaStream_t st);

struct AppendArgs {
  const void* in[2];     // k, v
  int64_t in_s[2][2];    // strides of head, token (elements)
  const int32_t* slot_map;
  const float* mean_k;   // [B, H_kv, d] or nullptr
  const int32_t* seq_ids;
  int T, B;
  sage_kv_cache_t c;
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st);

struct DecodeArgs {
  const void* q;
  int64_t q_s[3];        // strides of batch, head, query token (elements)
  sage_kv_cache_t c;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* o;
  float* lse;            // or nullptr
  void* ws;
  int max_pages, B, H, n_q, max_len, causal;
  float sm_scale;
  uint64_t timeout_ns;   // of the kernel's waits
};
size_t decode_workspace_bytes(int B, int H, int H_kv, int n_q, int d, int max_len, int format);
cudaError_t decode_read_and_clear_error(uint32_t* word);
cudaError_t launch_attn_decode(const DecodeArgs& a, cudaStream_t st);

}  // namespace sage
