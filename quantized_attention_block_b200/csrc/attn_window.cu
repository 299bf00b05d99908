// attn_window.cu -- sliding-window attention with sinks (16-bit, forward).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "serving.cuh"

namespace sage {

namespace {

constexpr int kRowWarps = 4;

// One row by one warp, over its visible keys alone: lane = key for the scores,
// lane = D / 32 channels for P V.
template <typename T, int D>
__device__ void window_row(const WindowArgs& a, int b, int hq, int i, float* s_q) {
  const int lane = threadIdx.x & 31;
  const int hk = hq / (a.Hq / a.Hkv);
  const int64_t qrow = row_offset((int64_t)b * a.Hq + hq, i, a.Hq, a.N, D, a.nhd);
  const int64_t krow = row_offset((int64_t)b * a.Hkv + hk, 0, a.Hkv, a.N, D, a.nhd);
  const int64_t ks = row_stride(a.Hkv, D, a.nhd);
  const T* k = static_cast<const T*>(a.k) + krow;
  const T* v = static_cast<const T*>(a.v) + krow;
  for (int d = lane; d < D; d += 32) s_q[d] = (float)static_cast<const T*>(a.q)[qrow + d];
  __syncwarp();
  const int ws = a.window > 0 && i + 1 > a.window ? i + 1 - a.window : 0;
  float m = -INFINITY, l = 0.0f, o[D / 32] = {};
  for (int part = 0; part < 2; ++part) {
    const int lo = part == 0 ? 0 : ws, hi = part == 0 ? min(a.sinks, ws) : i + 1;
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      float t = -INFINITY;
      if (j < hi) {
        const uint4* row = reinterpret_cast<const uint4*>(k + j * ks);
        float x = 0.0f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = row[c];
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<T>(u[e]);
            x = fmaf(f.x, s_q[c * 8 + 2 * e], x);
            x = fmaf(f.y, s_q[c * 8 + 2 * e + 1], x);
          }
        }
        t = x * a.scale_log2;
      }
      float mx = t;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.0f : mn;
      const float alpha = exp2f(m - ms), p = exp2f(t - ms);
      m = mn;
      float sum = p;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l = l * alpha + sum;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] *= alpha;
      const int n = min(32, hi - j0);
      for (int x = 0; x < n; ++x) {
        const float w = __shfl_sync(0xffffffffu, p, x);
        const uint32_t* row = reinterpret_cast<const uint32_t*>(v + (j0 + x) * ks) + lane * (D / 64);
#pragma unroll
        for (int d = 0; d < D / 64; ++d) {
          const float2 f = unpack2<T>(row[d]);
          o[2 * d] = fmaf(w, f.x, o[2 * d]);
          o[2 * d + 1] = fmaf(w, f.y, o[2 * d + 1]);
        }
      }
    }
  }
  const float inv = 1.0f / l;
  T* out = static_cast<T*>(a.o) + qrow + lane * (D / 32);
#pragma unroll
  for (int d = 0; d < D / 32; ++d) out[d] = (T)(o[d] * inv);
  if (a.lse && lane == 0) a.lse[((int64_t)b * a.Hq + hq) * a.N + i] = (m + log2f(l)) * 0.6931471805599453f;
  __syncwarp();
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kRowWarps) window_rows_kernel(const WindowArgs a) {
  __shared__ float s_q[kRowWarps][D];
  const int warp = threadIdx.x >> 5;
  const int64_t w = (int64_t)blockIdx.x * kRowWarps + warp;
  if (w >= (int64_t)a.B * a.Hq * a.N) return;
  const int i = (int)(w % a.N), bh = (int)(w / a.N);
  const int b = bh / a.Hq;
  if (a.lens && i >= min(max(a.lens[b], 0), a.N)) return;
  window_row<T, D>(a, b, bh % a.Hq, i, s_q[warp]);
}

}  // namespace

cudaError_t launch_attn_window(const WindowArgs& a, int is_fp16, cudaStream_t st) {
  const int64_t rows = (int64_t)a.B * a.Hq * a.N;
  const unsigned grid = (unsigned)((rows + kRowWarps - 1) / kRowWarps);
  if (a.D == 128) {
    if (is_fp16) window_rows_kernel<__half, 128><<<grid, 32 * kRowWarps, 0, st>>>(a);
    else window_rows_kernel<__nv_bfloat16, 128><<<grid, 32 * kRowWarps, 0, st>>>(a);
  } else {
    if (is_fp16) window_rows_kernel<__half, 64><<<grid, 32 * kRowWarps, 0, st>>>(a);
    else window_rows_kernel<__nv_bfloat16, 64><<<grid, 32 * kRowWarps, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace sage
