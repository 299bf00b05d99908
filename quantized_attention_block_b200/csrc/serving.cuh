// serving.cuh -- argument blocks and device helpers of the paged key-value
// cache, the single-token attention over it and the sliding-window attention.
#pragma once
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "sm100.cuh"

namespace sage {

constexpr int kBlk = 16;          // keys of one decode block (a page holds whole blocks)
constexpr int kDecodeCtas = 592;  // most CTAs (and half the partial slots) of one decode call
constexpr int kMaxGroup = 16;     // query heads of one decode row (an MMA's 16 rows)

struct CacheArgs {
  void* k;  // pages; element strides: page, head, row
  void* v;
  float* ks;  // [n_pages, H, page]
  float* vs;
  float* weight;
  int H, D, page_log2, n_pages;
  int64_t page_stride, hs, rs;
  const int* table;
  const int* lens;
  int B, max_pages;
  int cap;  // max_pages * page
};

struct AppendArgs {
  CacheArgs c;
  const void* k;
  const void* v;
  const int* n_new;  // nullptr: T
  const float* km;   // nullptr: zeros
  int T, nhd;
  int quantized, is_fp16;
};

struct DecodeArgs {
  CacheArgs c;
  const void* q;  // [B, Hq, D]
  void* o;
  float* lse;
  const float* km;
  int Hq, G, GT;  // query heads, heads a group, group tiles (of 8 or 16 heads)
  int window, sinks;
  int q_fp16;
  float scale_log2, sm_scale;
  int direct;  // a CTA a row of work, nothing to join (decode_direct)
  // workspace
  long long* prefix;  // [B] units before sequence b; [B] = units a CTA
  float* part_m;      // [2 kDecodeCtas][kMaxGroup]
  float* part_l;
  float* part_o;      // [2 kDecodeCtas][kMaxGroup][D]
  float* lse2;        // [B, Hq] log2-sum-exp2 (only with weights)
  float* scores;      // [B, Hq, score_cap] log2 scores of the visible blocks (only with weights)
  int64_t score_cap;
};

struct EvictArgs {
  CacheArgs c;
  const int* dst_table;
  int dst_pages;
  int keep, sinks, recent;
  int* new_lens;
  int* kept;
  int quantized;
  int held_keys;  // set at launch: weights that the selection keeps in shared memory
};

struct WindowArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  const int* lens;
  int B, Hq, Hkv, N, D;
  int nhd, window, sinks;
  int zero_tail;  // rows behind a sequence's end: 1 zeros into o, 2 into lse
  float sm_scale, scale_log2;
  int items, pairs, group;  // set at launch: work items, row pairs of a head, heads whose items follow one another
};

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st);
cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t st);
cudaError_t launch_attn_decode(const DecodeArgs& a, int quantized, cudaStream_t st);
cudaError_t launch_attn_window(const WindowArgs& a, int is_fp16, cudaStream_t st);

// ------------------------------------------------------------------ host
// What a launcher asks of the current device once (attributes of a kernel, its
// CTAs that run at a time): a call of microseconds has no time to ask again.
// Two threads may both ask; they get the same answer.
struct DeviceOnce {
  static constexpr int kDevices = 64;
  std::atomic<bool> done[kDevices] = {};
  std::atomic<int> value[kDevices] = {};  // what f(device) leaves there
  template <typename F>
  cudaError_t run(F&& f, int* got = nullptr) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {
      if ((e = f(dev)) != cudaSuccess) return e;
      done[dev].store(true, std::memory_order_release);
    }
    if (got) *got = value[dev];
    return cudaSuccess;
  }
};

// ------------------------------------------------------------------ cache
__device__ __forceinline__ void record_page_error() { atomicExch(&g_page_error, 1u); }

// tokens that sequence b holds, taken as the nearest bound if outside [0, cap]
__device__ __forceinline__ int cache_len(const CacheArgs& c, int b) { return min(max(c.lens[b], 0), c.cap); }

// The blocks of kBlk keys that a query at position n - 1 looks at: blocks
// [0, nsb) for the sinks, then [wb, ceil(n / kBlk)) for the window; a block of
// both belongs to the latter.  Keys are visible when j < n and (j >= ws or j < sinks).
struct Span {
  int n, ws, nsb, wb, vb;
};
__device__ __forceinline__ Span visible_span(int n, int window, int sinks) {
  Span s;
  s.n = n;
  s.ws = (window > 0 && n > window) ? n - window : 0;
  s.wb = s.ws / kBlk;
  s.nsb = min((min(sinks, s.ws) + kBlk - 1) / kBlk, s.wb);
  s.vb = s.nsb + (n + kBlk - 1) / kBlk - s.wb;
  return s;
}
// blocks that a query can look at, at most (cap: slots of a sequence)
inline int64_t most_blocks(int64_t cap, int window, int sinks) {
  const int64_t all = (cap + kBlk - 1) / kBlk;
  const int64_t seen = (int64_t)window / kBlk + 2 + ((int64_t)sinks + kBlk - 1) / kBlk;
  return window > 0 && seen < all ? seen : all;
}
// Whether a row of work of at most `blocks` blocks goes to one CTA: short ones (a split's second kernel
// costs more than the 8 turns of 4 warps), and those of up to four times the length when there are rows
// enough for every SM twice.
inline bool decode_direct(int64_t rows, int64_t blocks) { return blocks <= 32 || (blocks <= 128 && rows >= 296); }
__device__ __forceinline__ int span_block(const Span& s, int i) { return i < s.nsb ? i : s.wb + i - s.nsb; }

// ------------------------------------------------------------------ types
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// ------------------------------------------------------------------ programmatic dependent launch
// The next kernel of the stream may be set up while this one runs; it waits in
// pdl_wait() until this one has finished and its writes are visible.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename K, typename A>
inline cudaError_t launch_pdl(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace sage
