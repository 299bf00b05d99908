// kv_cache.cu -- the paged key-value cache: writing new tokens (16 bit, or INT8
// keys and E4M3 values with one scale per token and head) and eviction by
// gathered attention weight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "serving.cuh"

namespace sage {

namespace {

// ------------------------------------------------------------------ append
// A row (token, head) of K and of V is D / 8 lanes of 16 bytes each.  Rows are
// taken in the order of the input, so reads are contiguous; a row lands
// contiguous in its page.  Bound: HBM (each token read and written once), so a
// thread holds its 16 bytes of K and V of ROWS rows at a time: the loads of
// ROWS = 4 are 128 bytes in flight a thread (prompts of 18k tokens of 8 heads of
// 128: 66 us with one row of K or V a thread).  Few rows take ROWS = 1, to be
// spread over more SMs.
constexpr int kAppendThreads = 256;

template <int D, bool QUANT, bool FP16, int ROWS>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
  constexpr int L = D / 8, PASS = kAppendThreads / L;  // lanes a row; rows of the CTA at a time
  const int lane = threadIdx.x % L, b = blockIdx.y;
  const uint32_t rows = (uint32_t)a.T * a.c.H, inner = a.nhd ? a.c.H : a.T;
  const int n_new = a.n_new ? min(max(__ldg(a.n_new + b), 0), a.T) : a.T;
  const int held = cache_len(a.c, b), page = 1 << a.c.page_log2;
  if (n_new > 0 && blockIdx.x == 0 && threadIdx.x == 0 &&
      (a.c.lens[b] != held || (int64_t)held + n_new > a.c.cap))
    record_page_error();
  // this thread's rows: (h, t), whether they are written (the lanes of a row agree, so shuffles below are among
  // active lanes), their place
  bool live[ROWS];
  int h[ROWS], off[ROWS], pid[ROWS];
  uint4 x[ROWS][2];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const uint32_t r = blockIdx.x * (ROWS * PASS) + i * PASS + threadIdx.x / L;
    const uint32_t q = r / inner, m = r - q * inner;
    const int t = a.nhd ? q : m;
    h[i] = a.nhd ? m : q;
    live[i] = r < rows && t < n_new && (uint32_t)held + (uint32_t)t < (uint32_t)a.c.cap;
    pid[i] = off[i] = 0;
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (live[i]) {
      const int64_t at = ((int64_t)b * rows + r) * L + lane;
      x[i][0] = __ldcs(static_cast<const uint4*>(a.k) + at);
      x[i][1] = __ldcs(static_cast<const uint4*>(a.v) + at);
      pid[i] = __ldg(a.c.table + (int64_t)b * a.c.max_pages + ((held + t) >> a.c.page_log2));
      off[i] = (held + t) & (page - 1);
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (live[i] && (uint32_t)pid[i] >= (uint32_t)a.c.n_pages) {
      record_page_error();
      live[i] = false;
    }
    const int64_t at = (int64_t)pid[i] * a.c.page_stride + h[i] * a.c.hs + off[i] * a.c.rs + lane * 8;
    const int64_t sat = ((int64_t)pid[i] * a.c.H + h[i]) * page + off[i];
    if (live[i] && lane == 0 && a.c.weight) a.c.weight[sat] = 0.0f;
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
      if constexpr (!QUANT) {
        if (live[i]) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + at) = x[i][is_v];
      } else {
        using T = std::conditional_t<FP16, __half, __nv_bfloat16>;
        float f[8];
        const uint32_t w[4] = {x[i][is_v].x, x[i][is_v].y, x[i][is_v].z, x[i][is_v].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p = unpack2<T>(w[e]);
          f[2 * e] = p.x;
          f[2 * e + 1] = p.y;
        }
        if (!is_v && a.km && live[i]) {
          const float4* km = reinterpret_cast<const float4*>(a.km + ((int64_t)b * a.c.H + h[i]) * D + lane * 8);
          const float4 m0 = __ldg(km), m1 = __ldg(km + 1);
          const float m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __fsub_rn(f[e], m[e]);
        }
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(f[e]));
#pragma unroll
        for (int m = L / 2; m > 0; m >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        const float s = __fdiv_rn(amax, is_v ? 448.0f : 127.0f);
        uint32_t lo = 0, hi = 0;
        if (s != 0.0f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __fdiv_rn(f[e], s);
          if (is_v) {
            lo = cvt_e4m3x4(f[0], f[1], f[2], f[3]);
            hi = cvt_e4m3x4(f[4], f[5], f[6], f[7]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int c = min(max(__float2int_rn(f[e]), -127), 127);
              (e < 4 ? lo : hi) |= (uint32_t)(c & 255) << (8 * (e & 3));
            }
          }
        }
        if (live[i]) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + at) = make_uint2(lo, hi);
          if (lane == 0) (is_v ? a.c.vs : a.c.ks)[sat] = s;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ evict
// Selection: one CTA per (b, kv head).  The weights' order-preserving bit
// patterns are searched for the (keep - sinks - recent)-th largest, 11 bits a
// pass (the first digit, sign, exponent and two bits, spreads weights over more
// than a handful of counters); a last pass in token order counts what stays and
// writes its positions.  The first pass keeps the patterns in shared memory
// (those of the first kSelKeys tokens; the others are looked up again): a pass
// through the page table took 30 us at 32k tokens, one over shared memory 3.
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelKeys = 53248;  // 208 KB

// unsigned key in the order of the weights: NaN lowest, -0 as +0
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t token_key(const CacheArgs& c, int b, int h, int j) {
  const int pid = __ldg(c.table + (int64_t)b * c.max_pages + (j >> c.page_log2));
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
  extern __shared__ __align__(16) uint32_t s_keys[];  // candidates [0, min(hi - lo, held))
  __shared__ int s_hist[kSelBins];
  __shared__ int s_warp[32], s_tie[kSelWarps], s_stay[kSelWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  pdl_launch();
  const int b = blockIdx.x / a.c.H, h = blockIdx.x % a.c.H, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int n = cache_len(a.c, b);
  if (h == 0 && tid == 0) {
    if (a.c.lens[b] != n) record_page_error();
    a.new_lens[b] = min(n, a.keep);
  }
  int* kept = a.kept + (int64_t)blockIdx.x * a.keep;
  if (n <= a.keep) {
    // (unsigned: the last step may pass 2^31)
    for (uint32_t i = tid; i < (uint32_t)a.keep; i += kSelThreads) kept[i] = i < (uint32_t)n ? (int)i : -1;
    return;
  }
  const int lo = a.sinks, cand = n - a.recent - lo;  // candidates: tokens lo + [0, cand)
  const int need = a.keep - a.sinks - a.recent;      // of them stay
  const int held = min(cand, a.held_keys);
  auto key_of = [&](int i) { return i < held ? s_keys[i] : token_key(a.c, b, h, lo + i); };
  uint32_t prefix = 0;
  int left = need;  // how many of the keys that match the prefix so far stay
  for (int pass = 0; pass < 3 && need > 0; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kSelBins;
    for (int i = tid; i < bins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    if (pass == 0) {
      for (int i0 = tid; i0 < cand; i0 += 4 * kSelThreads) {
        uint32_t k[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = i0 + x * kSelThreads;
          if (i < cand) k[x] = token_key(a.c, b, h, lo + i);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = i0 + x * kSelThreads;
          if (i < held) s_keys[i] = k[x];
          if (i < cand) atomicAdd(&s_hist[k[x] >> 21], 1);
        }
      }
    } else {
      for (int i = tid; i < cand; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if (k >> (pass == 1 ? 21 : 10) == prefix) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1);
      }
    }
    __syncthreads();
    // the digit at which the count from the largest down reaches `left`; two bins a thread
    const int i1 = bins - 1 - 2 * tid, i0 = i1 - 1;
    const int x1 = i0 >= 0 ? s_hist[i1] : 0, x0 = i0 >= 0 ? s_hist[i0] : 0;
    int total;
    const int before = block_scan(x1 + x0, s_warp, &total);
    if (before < left && left <= before + x1 + x0) {
      const bool first = left <= before + x1;
      s_prefix = (prefix << (pass == 2 ? 10 : 11)) | (first ? i1 : i0);
      s_need = left - before - (first ? 0 : x1);
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_need;
    __syncthreads();
  }
  // `left` of the keys equal to `prefix` stay, the earliest.  A warp takes a run of tokens, 32 at a time: it counts
  // the larger and the equal ones, then, with the counts of the warps before it, writes the positions.
  const int run = ((cand + kSelThreads - 1) / kSelThreads) * 32;
  const int i0 = warp * run, i1 = min(cand, i0 + run);
  int more = 0, same = 0;
  if (need > 0)
    for (int i = i0; i < i1; i += 32) {
      const uint32_t k = i + lane < i1 ? key_of(i + lane) : 0u;
      more += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && k > prefix));
      same += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && k == prefix));
    }
  if (lane == 0) {
    s_stay[warp] = more;
    s_tie[warp] = same;
  }
  __syncthreads();
  int out = a.sinks, ties = 0;
  for (int w = 0; w < warp; ++w) {
    out += s_stay[w] + max(0, min(s_tie[w], left - ties));
    ties += s_tie[w];
  }
  if (need > 0)
    for (int i = i0; i < i1; i += 32) {
      const uint32_t k = i + lane < i1 ? key_of(i + lane) : 0u;
      const uint32_t tie = __ballot_sync(0xffffffffu, i + lane < i1 && k == prefix);
      const uint32_t below = (1u << lane) - 1u;
      const bool stay = i + lane < i1 && (k > prefix || (k == prefix && ties + __popc(tie & below) < left));
      const uint32_t all = __ballot_sync(0xffffffffu, stay);
      if (stay) kept[out + __popc(all & below)] = lo + i + lane;
      out += __popc(all);
      ties += __popc(tie);
    }
  for (int i = tid; i < a.sinks; i += kSelThreads) kept[i] = i;
  for (int i = tid; i < a.recent; i += kSelThreads) kept[a.keep - a.recent + i] = n - a.recent + i;
}

// Moves the rows that stay.  One row of K or V is ROW_BYTES / 16 lanes; a thread
// has its 16 bytes of K and V of two rows in flight.  More are slower, not faster
// (192 us on the device for the whole call with two, 246 with four, 321 with eight,
// for 128 rows of up to 12288 tokens), and so are accesses that stay in L2 (212 us).
// (With the weights and scales moved as below, 180.)
// (kept with plain loads: the selection may still write it when this kernel
// starts, and the non-coherent ones are for data that no kernel writes meanwhile.)
constexpr int kMoveThreads = 128, kMoveRows = 2;

template <int ROW_BYTES>
__global__ void __launch_bounds__(kMoveThreads) kv_move_kernel(const EvictArgs a) {
  pdl_wait();
  constexpr int L = ROW_BYTES / 16;
  constexpr int PASS = kMoveThreads / L;  // rows of the CTA at a time
  const int bh = blockIdx.x, b = bh / a.c.H, h = bh % a.c.H;
  const int n = min(cache_len(a.c, b), a.keep);
  const int lane = threadIdx.x % L;
  const int page = 1 << a.c.page_log2;
  const int esize = a.quantized ? 1 : 2;
  // weights and scales, a thread a row (by a lane of each row's in the loop below, 198 us a call against 190 for 128
  // rows of up to 12288 tokens; on the device 192 and 180; bad pages are recorded there)
  constexpr int ROWS = PASS * kMoveRows;  // of the CTA at a time
  static_assert(ROWS <= kMoveThreads, "a thread a row");
  for (int i = blockIdx.y * ROWS + threadIdx.x; threadIdx.x < ROWS && i < n; i += gridDim.y * ROWS) {
    const int j = a.kept[(int64_t)bh * a.keep + i];
    const int sp = __ldg(a.c.table + (int64_t)b * a.c.max_pages + (j >> a.c.page_log2));
    const int dp = __ldg(a.dst_table + (int64_t)b * a.dst_pages + (i >> a.c.page_log2));
    if ((uint32_t)sp >= (uint32_t)a.c.n_pages || (uint32_t)dp >= (uint32_t)a.c.n_pages) continue;
    const int64_t ss = ((int64_t)sp * a.c.H + h) * page + (j & (page - 1));
    const int64_t ds = ((int64_t)dp * a.c.H + h) * page + (i & (page - 1));
    const float w = a.c.weight[ss];
    if (a.quantized) {
      const float x = a.c.ks[ss], y = a.c.vs[ss];
      a.c.ks[ds] = x;
      a.c.vs[ds] = y;
    }
    a.c.weight[ds] = w;
  }
  for (int i0 = blockIdx.y * ROWS + threadIdx.x / L; i0 < n; i0 += gridDim.y * ROWS) {
    int j[kMoveRows], sp[kMoveRows], dp[kMoveRows];
    uint4 kx[kMoveRows], vx[kMoveRows];
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
      const int i = i0 + x * PASS;
      j[x] = i < n ? a.kept[(int64_t)bh * a.keep + i] : -1;
      dp[x] = i < n ? __ldg(a.dst_table + (int64_t)b * a.dst_pages + (i >> a.c.page_log2)) : 0;
    }
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x)
      sp[x] = j[x] >= 0 ? __ldg(a.c.table + (int64_t)b * a.c.max_pages + (j[x] >> a.c.page_log2)) : 0;
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
      if (j[x] < 0) continue;
      if ((uint32_t)sp[x] >= (uint32_t)a.c.n_pages || (uint32_t)dp[x] >= (uint32_t)a.c.n_pages) {
        record_page_error();
        j[x] = -1;
        continue;
      }
      const int so = j[x] & (page - 1);
      const int64_t src = ((int64_t)sp[x] * a.c.page_stride + h * a.c.hs + so * a.c.rs) * esize + lane * 16;
      kx[x] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c.k) + src));
      vx[x] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.c.v) + src));
    }
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
      if (j[x] < 0) continue;
      const int to = (i0 + x * PASS) & (page - 1);
      const int64_t dst = ((int64_t)dp[x] * a.c.page_stride + h * a.c.hs + to * a.c.rs) * esize + lane * 16;
      __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.c.k) + dst), kx[x]);
      __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.c.v) + dst), vx[x]);
    }
  }
}

template <int D, bool QUANT, bool FP16>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t st) {
  constexpr int PASS = kAppendThreads / (D / 8);
  const int64_t rows = (int64_t)a.T * a.c.H;
  // four rows a thread once that leaves every SM a few CTAs
  if (rows * a.c.B >= (int64_t)4 * PASS * 148 * 4) {
    const dim3 grid((unsigned)((rows + 4 * PASS - 1) / (4 * PASS)), (unsigned)a.c.B);
    kv_append_kernel<D, QUANT, FP16, 4><<<grid, kAppendThreads, 0, st>>>(a);
  } else {
    const dim3 grid((unsigned)((rows + PASS - 1) / PASS), (unsigned)a.c.B);
    kv_append_kernel<D, QUANT, FP16, 1><<<grid, kAppendThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  if (a.c.D == 128) {
    if (!a.quantized) return launch_append_t<128, false, false>(a, st);
    return a.is_fp16 ? launch_append_t<128, true, true>(a, st) : launch_append_t<128, true, false>(a, st);
  }
  if (!a.quantized) return launch_append_t<64, false, false>(a, st);
  return a.is_fp16 ? launch_append_t<64, true, true>(a, st) : launch_append_t<64, true, false>(a, st);
}

cudaError_t launch_kv_evict(const EvictArgs& args, cudaStream_t st) {
  EvictArgs a = args;
  const int rows = a.c.B * a.c.H;
  static DeviceOnce once;
  cudaError_t e = once.run([&](int) {
    return cudaFuncSetAttribute(kv_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kSelKeys);
  });
  if (e != cudaSuccess) return e;
  // room for the keys of the longest sequence that the table can hold: less lets more CTAs share an SM
  const int64_t most = (int64_t)a.c.cap - a.sinks - a.recent;
  a.held_keys = (int)(most < 0 ? 0 : most > kSelKeys ? kSelKeys : most);
  kv_select_kernel<<<rows, kSelThreads, (size_t)4 * a.held_keys, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int row_bytes = a.c.D * (a.quantized ? 1 : 2);
  const int rpc = kMoveThreads / (row_bytes / 16) * kMoveRows;
  const int64_t want = ((int64_t)a.keep + rpc - 1) / rpc;
  const dim3 grid((unsigned)rows, (unsigned)(want < 65535 ? want : 65535));
  switch (row_bytes) {
    case 256: return launch_pdl(kv_move_kernel<256>, grid, dim3(kMoveThreads), 0, st, a);
    case 128: return launch_pdl(kv_move_kernel<128>, grid, dim3(kMoveThreads), 0, st, a);
    default: return launch_pdl(kv_move_kernel<64>, grid, dim3(kMoveThreads), 0, st, a);
  }
}

}  // namespace sage
