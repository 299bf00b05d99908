// kv_cache.cu -- the paged key-value cache: writing new tokens (16 bit, or INT8
// keys and E4M3 values with one scale per token and head) and eviction by
// gathered attention weight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "serving.cuh"

namespace sage {

namespace {

// ------------------------------------------------------------------ append
// One row (token, head) of K or V is D / 8 lanes of 16 bytes.  Rows are taken
// in the order of the input, so reads are contiguous; a row lands contiguous in
// its page.  Bound: HBM (each token read and written once).
constexpr int kAppendThreads = 256;

template <int D, bool QUANT, bool FP16>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
  constexpr int L = D / 8;  // lanes a row
  const int64_t rows = (int64_t)a.c.B * a.T * a.c.H;
  const int lane = threadIdx.x % L;
  const int64_t row = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) / L;
  const bool is_v = blockIdx.y != 0;
  const int page = 1 << a.c.page_log2;
  // (b, h, t) of the row; the lanes of a row agree, so shuffles below are among active lanes
  bool live = row < rows;
  const int64_t r = live ? row : 0;
  const int inner = (int)(r % (a.nhd ? a.c.H : a.T));
  const int64_t outer = r / (a.nhd ? a.c.H : a.T);
  const int mid = (int)(outer % (a.nhd ? a.T : a.c.H));
  const int b = (int)(outer / (a.nhd ? a.T : a.c.H));
  const int h = a.nhd ? inner : mid, t = a.nhd ? mid : inner;
  const int n_new = a.n_new ? min(max(a.n_new[b], 0), a.T) : a.T;
  live = live && t < n_new;
  int pos = 0, pid = 0;
  if (live) {
    const int64_t p = (int64_t)cache_len(a.c, b) + t;
    if (p >= a.c.cap || a.c.lens[b] < 0 || a.c.lens[b] > a.c.cap) record_page_error();
    live = p < a.c.cap;
    pos = (int)p;
  }
  if (live) {
    pid = a.c.table[(int64_t)b * a.c.max_pages + (pos >> a.c.page_log2)];
    if (pid < 0 || pid >= a.c.n_pages) {
      record_page_error();
      live = false;
    }
  }
  uint4 x = make_uint4(0, 0, 0, 0);
  if (live) x = reinterpret_cast<const uint4*>(is_v ? a.v : a.k)[r * L + lane];
  const int off = pos & (page - 1);
  const int64_t at = (int64_t)pid * a.c.page_stride + h * a.c.hs + off * a.c.rs + lane * 8;
  const int64_t sat = ((int64_t)pid * a.c.H + h) * page + off;
  if (live && lane == 0 && !is_v && a.c.weight) a.c.weight[sat] = 0.0f;
  if constexpr (!QUANT) {
    if (live) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + at) = x;
  } else {
    using T = std::conditional_t<FP16, __half, __nv_bfloat16>;
    float f[8];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack2<T>(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
    if (!is_v && a.km) {
      const float* km = a.km + ((int64_t)b * a.c.H + h) * D + lane * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __fsub_rn(f[i], km[i]);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(f[i]));
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    const float s = __fdiv_rn(amax, is_v ? 448.0f : 127.0f);
    uint32_t lo = 0, hi = 0;
    if (s != 0.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], s);
      if (is_v) {
        lo = cvt_e4m3x4(f[0], f[1], f[2], f[3]);
        hi = cvt_e4m3x4(f[4], f[5], f[6], f[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = min(max(__float2int_rn(f[i]), -127), 127);
          (i < 4 ? lo : hi) |= (uint32_t)(c & 255) << (8 * (i & 3));
        }
      }
    }
    if (live) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + at) = make_uint2(lo, hi);
      if (lane == 0) (is_v ? a.c.vs : a.c.ks)[sat] = s;
    }
  }
}

// ------------------------------------------------------------------ evict
// Selection: one CTA per (b, kv head).  The weights' order-preserving bit
// patterns are searched for the (keep - sinks - recent)-th largest, 8 bits a
// pass; a last pass in token order counts what stays and writes its positions.
constexpr int kSelThreads = 1024;

// unsigned key in the order of the weights: NaN lowest, -0 as +0
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t token_key(const CacheArgs& c, int b, int h, int j) {
  const int pid = c.table[(int64_t)b * c.max_pages + (j >> c.page_log2)];
  if (pid < 0 || pid >= c.n_pages) {
    record_page_error();
    return 0u;
  }
  const int page = 1 << c.page_log2;
  return weight_key(c.weight[((int64_t)pid * c.H + h) * page + (j & (page - 1))]);
}

// exclusive sum of x over the CTA's threads; *total: the sum of all
__device__ __forceinline__ int block_scan(int x, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return v - x + (warp ? s_warp[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const EvictArgs a) {
  __shared__ int s_hist[256];
  __shared__ int s_warp[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int b = blockIdx.x / a.c.H, h = blockIdx.x % a.c.H, tid = threadIdx.x;
  const int n = cache_len(a.c, b);
  if (h == 0 && tid == 0) {
    if (a.c.lens[b] != n) record_page_error();
    a.new_lens[b] = min(n, a.keep);
  }
  int* kept = a.kept + (int64_t)blockIdx.x * a.keep;
  if (n <= a.keep) {
    for (int i = tid; i < a.keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int lo = a.sinks, hi = n - a.recent;  // candidates [lo, hi)
  const int need = a.keep - a.sinks - a.recent;
  uint32_t prefix = 0;
  int left = need;  // how many of the keys that match the prefix so far stay
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t key = token_key(a.c, b, h, j);
      if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&s_hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    int total;
    const int x = tid < 256 ? s_hist[255 - tid] : 0;  // from the largest digit down
    const int before = block_scan(x, s_warp, &total);
    if (tid < 256 && before < left && left <= before + x) {
      s_prefix = (prefix << 8) | (255 - tid);
      s_need = left - before;
    }
    __syncthreads();
    if (left > 0) {
      prefix = s_prefix;
      left = s_need;
    }
    __syncthreads();
  }
  // `left` of the keys equal to `prefix` stay (the earliest); need == 0: none at all
  int out = 0, ties = 0;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + tid;
    bool stay = false, tie = false;
    if (j < n) {
      if (j < lo || j >= hi) {
        stay = true;
      } else if (need > 0) {
        const uint32_t key = token_key(a.c, b, h, j);
        stay = key > prefix;
        tie = key == prefix;
      }
    }
    int total;
    const int tie_rank = ties + block_scan(tie ? 1 : 0, s_warp, &total);
    ties += total;
    stay = stay || (tie && tie_rank < left);
    const int at = out + block_scan(stay ? 1 : 0, s_warp, &total);
    out += total;
    if (stay && at < a.keep) kept[at] = j;
  }
}

// Moves the rows that stay.  One row of K or V is D * bytes / 16 lanes.
constexpr int kMoveThreads = 256;

template <int ROW_BYTES>
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const EvictArgs a) {
  pdl_wait();
  constexpr int L = ROW_BYTES / 16;
  constexpr int RPC = kMoveThreads / L;  // rows a CTA pass
  const int bh = blockIdx.x, b = bh / a.c.H, h = bh % a.c.H;
  const int n = min(cache_len(a.c, b), a.keep);
  const int lane = threadIdx.x % L;
  const int page = 1 << a.c.page_log2;
  const int esize = a.quantized ? 1 : 2;
  for (int i = blockIdx.y * RPC + threadIdx.x / L; i < n; i += gridDim.y * RPC) {
    const int j = a.kept[(int64_t)bh * a.keep + i];
    const int sp = a.c.table[(int64_t)b * a.c.max_pages + (j >> a.c.page_log2)];
    const int dp = a.dst_table[(int64_t)b * a.dst_pages + (i >> a.c.page_log2)];
    if (sp < 0 || sp >= a.c.n_pages || dp < 0 || dp >= a.c.n_pages) {
      record_page_error();
      continue;
    }
    const int so = j & (page - 1), to = i & (page - 1);
    const int64_t src = ((int64_t)sp * a.c.page_stride + h * a.c.hs + so * a.c.rs) * esize + lane * 16;
    const int64_t dst = ((int64_t)dp * a.c.page_stride + h * a.c.hs + to * a.c.rs) * esize + lane * 16;
    const uint4 kx = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c.k) + src);
    const uint4 vx = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c.v) + src);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.c.k) + dst) = kx;
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.c.v) + dst) = vx;
    const int64_t ss = ((int64_t)sp * a.c.H + h) * page + so, ds = ((int64_t)dp * a.c.H + h) * page + to;
    if (lane == 0) a.c.weight[ds] = a.c.weight[ss];
    if (a.quantized && lane == 1) a.c.ks[ds] = a.c.ks[ss];
    if (a.quantized && lane == 2) a.c.vs[ds] = a.c.vs[ss];
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
  const int L = a.c.D / 8;
  const int64_t rows = (int64_t)a.c.B * a.T * a.c.H;
  const dim3 grid((unsigned)((rows * L + kAppendThreads - 1) / kAppendThreads), 2);
  if (rows == 0) return cudaSuccess;
  if (a.c.D == 128) {
    if (!a.quantized) kv_append_kernel<128, false, false><<<grid, kAppendThreads, 0, st>>>(a);
    else if (a.is_fp16) kv_append_kernel<128, true, true><<<grid, kAppendThreads, 0, st>>>(a);
    else kv_append_kernel<128, true, false><<<grid, kAppendThreads, 0, st>>>(a);
  } else {
    if (!a.quantized) kv_append_kernel<64, false, false><<<grid, kAppendThreads, 0, st>>>(a);
    else if (a.is_fp16) kv_append_kernel<64, true, true><<<grid, kAppendThreads, 0, st>>>(a);
    else kv_append_kernel<64, true, false><<<grid, kAppendThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t st) {
  const int rows = a.c.B * a.c.H;
  kv_select_kernel<<<rows, kSelThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int row_bytes = a.c.D * (a.quantized ? 1 : 2);
  const int rpc = kMoveThreads / (row_bytes / 16);
  const int want = (a.keep + rpc - 1) / rpc;
  const dim3 grid((unsigned)rows, (unsigned)(want < 65535 ? want : 65535));
  switch (row_bytes) {
    case 256: return launch_pdl(kv_move_kernel<256>, grid, dim3(kMoveThreads), 0, st, a);
    case 128: return launch_pdl(kv_move_kernel<128>, grid, dim3(kMoveThreads), 0, st, a);
    default: return launch_pdl(kv_move_kernel<64>, grid, dim3(kMoveThreads), 0, st, a);
  }
}

}  // namespace sage
