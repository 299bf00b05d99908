// decode.cu -- attention of one new token over the paged key-value cache, split
// over the cache's length and joined.
//
// Per query head, over the visible keys j (serving.cuh: Span):
//   t_j = sm_scale log2(e) q . K_j,  m = max t,  l = sum 2^(t_j - m),
//   o = sum 2^(t_j - m) V_j / l,     lse = (m + log2 l) ln 2
// and, with weights, weight[j] += sum over the group's heads of 2^(t_j - m) / l.
//
// Bound: HBM, each visible K and V row read once.  A row of work is a
// (sequence, kv head, tile of up to 16 of its query heads); the blocks of 16
// keys of all rows in one line are cut into equal shares, one a CTA, whatever
// the lengths are, so the lengths stay on the device and a captured graph
// serves any of them.  A CTA's share covers at most one row it shares with the
// CTA before it and one with the CTA after: two slots of partial results a CTA,
// joined in the order of the CTAs by a second kernel (no atomics: the same
// inputs give the same bytes).
//
// A warp takes every fourth block of a piece with a ring of its own in shared
// memory (cp.async, no CTA barrier in the loop) and keeps its own m, l and O;
// the four warps are merged at the end of the piece.  Rows that are not visible
// are not read: cp.async fills them with zeros, so nothing an unused slot holds
// (NaN) can reach a sum.
//
// mma.sync m16n8k16 rather than tcgen05: the 16 rows of A are the group's query
// heads, and at 24 B a clock and SM of HBM the tensor work is a few per cent of
// either pipe; fragments in registers save the round trip through TMEM.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "serving.cuh"

namespace sage {

namespace {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kMinShare = 8;  // blocks of the smallest share: two a warp (4k tokens of 8 heads: 14.0 us with 4, 12.7 with 8, 13.8 with 16)

enum CacheType : int { kBF16 = 0, kFP16 = 1, kQ8 = 2 };

template <int D, int CT>
struct DecTile {
  static constexpr int kRow = D * (CT == kQ8 ? 1 : 2);                   // bytes of a row of K or V
  static constexpr int kBlkBytes = kBlk * kRow;
  static constexpr int kStage = 2 * kBlkBytes + (CT == kQ8 ? 128 : 0);   // K, V, 16 + 16 scales
  // blocks in the ring, the one worked on among them: one of 8 KB of K and V on the way, or two smaller ones (64 x 12k
  // tokens of 16 bits and d = 128: 277 us with 3, 272 with 2; 131k tokens in 8 bit: 62 us with 3, 65 with 2)
  static constexpr int kStages = kBlkBytes >= 4096 ? 2 : 3;
  static constexpr int kWarpBytes = kStages * kStage;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool pred) {
  const int n = pred ? 16 : 0;  // 0: fills with zeros, reads nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// a cached row is read once a call: first out of L2 (64 x 12k tokens: 284 -> 277 us, 131k in 8 bit: 65 -> 62 us)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16-byte chunk c of row r of a tile with `ROW` bytes a row: rows of one
// 8-row matrix land in different banks
template <int ROW>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  constexpr int C = ROW / 16;
  return r * ROW + 16 * (C >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3));
}

// two INT8 pairs of a word -> fp16 pairs (exact): code + 128 under the exponent
// of 1024, minus 1152
__device__ __forceinline__ void int8x4_to_half(uint32_t x, uint32_t& p01, uint32_t& p23) {
  x ^= 0x80808080u;
  const uint32_t lo = __byte_perm(x, 0x64646464u, 0x4140), hi = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 off = __floats2half2_rn(1152.0f, 1152.0f);
  __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), off);
  __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
  p01 = *reinterpret_cast<uint32_t*>(&a);
  p23 = *reinterpret_cast<uint32_t*>(&b);
}

// the E4M3 codes in bytes (0, 2) and (1, 3) of a word -> fp16 pairs (exact)
__device__ __forceinline__ void e4m3x4_to_half(uint32_t x, uint32_t& even, uint32_t& odd) {
  const uint32_t y = __byte_perm(x, x, 0x3120);
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(even), "=r"(odd)
      : "r"(y));
}

// a pair of fp32 weights as 16-bit numbers, and what that rounding left over
template <bool BF16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  }
}

template <typename T>
__device__ __forceinline__ T to16(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 to16<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half to16<__half>(float x) { return __float2half_rn(x); }

__device__ __forceinline__ void store16(void* o, int64_t i, float x, int fp16) {
  if (fp16) static_cast<__half*>(o)[i] = to16<__half>(x);
  else static_cast<__nv_bfloat16*>(o)[i] = to16<__nv_bfloat16>(x);
}
__device__ __forceinline__ float load16(const void* p, int64_t i, int fp16) {
  return fp16 ? __half2float(static_cast<const __half*>(p)[i]) : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// A warp writes one head's log-sum-exp (m, l in base 2), with the shift by km
template <int D>
__device__ __forceinline__ void write_lse(const DecodeArgs& a, int b, int hq, float m, float l) {
  const int lane = threadIdx.x & 31;
  const bool some = l > 0.0f || isnan(l);  // (without a key: -inf, whatever the query of a padded row holds)
  const float lse2 = some ? m + log2f(l) : -INFINITY;
  float dot = 0.0f;
  if (a.km && a.lse && some) {
    const float* km = a.km + ((int64_t)b * a.c.H + hq / a.G) * D;
    for (int i = lane; i < D; i += 32) dot += load16(a.q, ((int64_t)b * a.Hq + hq) * D + i, a.q_fp16) * km[i];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
  }
  if (lane == 0) {
    if (a.lse) a.lse[(int64_t)b * a.Hq + hq] = lse2 * 0.6931471805599453f + a.sm_scale * dot;
    if (a.lse2) a.lse2[(int64_t)b * a.Hq + hq] = lse2;
  }
}

// weight of the visible slots first, first + stride, ... of (b, h) += sum over the group's heads of 2^(t - lse2);
// four at a time, so that their page numbers and weights are on the way together (9 of 26 us one by one, for
// 384 heads that see 1028 keys)
template <typename F>
__device__ __forceinline__ void add_weights(const DecodeArgs& a, const Span& sp, int b, int h, int first, int stride,
                                            F lse2) {
  constexpr int U = 4;
  const int page = 1 << a.c.page_log2, end = sp.vb * kBlk;
  const float* scores = a.scores + ((int64_t)b * a.Hq + h * a.G) * a.score_cap;
  for (int i0 = first; i0 < end; i0 += U * stride) {
    int j[U], pid[U];
    float* w[U];
    float x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + k * stride;
      j[k] = i < end ? span_block(sp, i / kBlk) * kBlk + i % kBlk : sp.n;
      if (j[k] >= sp.n || (j[k] < sp.ws && j[k] >= a.sinks)) pid[k] = -1;
      else pid[k] = __ldg(a.c.table + (int64_t)b * a.c.max_pages + (j[k] >> a.c.page_log2));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      w[k] = nullptr;
      x[k] = 0.0f;
      if ((uint32_t)pid[k] < (uint32_t)a.c.n_pages) {
        w[k] = a.c.weight + ((int64_t)pid[k] * a.c.H + h) * page + (j[k] & (page - 1));
        x[k] = *w[k];
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (!w[k]) continue;
      const float* t = scores + i0 + k * stride;
      float y = 0.0f;
      for (int g = 0; g < a.G; ++g) y += exp2f(t[g * a.score_cap] - lse2(g));
      *w[k] = x[k] + y;
    }
  }
}

// register i of Q's fragment; with 8 heads a row, rows 8-15 are zeros
template <int MT, int I, int N>
__device__ __forceinline__ uint32_t q_frag(const uint32_t (&q)[N]) {
  if constexpr (MT == 16) return q[I];
  else if constexpr (I == 2) return q[1];
  else return 0u;
}

// MT: query heads of a row of work (8: rows 8-15 of the MMA's A carry the low
// halves of the weights; 16: a second MMA does)
// SPLIT: the shares described above; else a CTA does one row of work alone, with
// the weights of its keys, and nothing is joined (see decode_direct)
template <int D, int CT, int MT, bool SPLIT>
__global__ void __launch_bounds__(kDecThreads) decode_kernel(const DecodeArgs a) {
  using Tile = DecTile<D, CT>;
  constexpr int kRow = Tile::kRow, S = Tile::kStages;
  constexpr int kLoads = Tile::kBlkBytes / 512;    // cp.async of one warp for a block of K or V
  constexpr int kChunks = kRow / 16;
  constexpr int kRowsPerLoad = 32 / kChunks;
  constexpr int NT = D / 8;                        // n-tiles of O
  constexpr bool kVB = CT == kBF16;                // V and the weights as bf16
  // fp16 weights (at most 1) are held in units of 2^-15: fp16 ends at 2^-24, and a weight of 2^-25 beside a heavy key
  // would be lost from O and kept in l.  (bf16 has fp32's range, and the 8-bit path a unit of its own, v_unit.)
  constexpr float kUnit = CT == kFP16 ? 32768.0f : 1.0f;
  constexpr int E = CT == kQ8 ? 1 : 2;             // bytes of an element
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_sum[kDecWarps];
  __shared__ long long s_base, s_off;
  __shared__ int s_b;
  __shared__ float s_m[kDecWarps][MT], s_l[kDecWarps][MT], s_lse[MT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int HG = a.c.H * a.GT;
  const int page_mask = (1 << a.c.page_log2) - 1;
  int b;
  long long off, u, u_end;  // the share: blocks [u, u_end), the first one `off` blocks into sequence b
  bool first_piece = true;
  if constexpr (SPLIT) {
    pdl_launch();
    // ---- this CTA's share of all blocks
    long long mine = 0;
    for (int seq = tid; seq < a.c.B; seq += kDecThreads) {
      const int n = cache_len(a.c, seq);
      if (blockIdx.x == 0 && a.c.lens[seq] != n) record_page_error();
      mine += visible_span(n, a.window, a.sinks).vb;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, x);
    if (lane == 0) s_sum[warp] = mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) total += s_sum[w];
    total *= HG;
    const long long share = max((long long)kMinShare, (total + gridDim.x - 1) / gridDim.x);
    u = blockIdx.x * share;
    u_end = min(total, u + share);
    if (blockIdx.x == 0 && tid == 0) a.prefix[a.c.B] = share;
    if (u >= u_end && blockIdx.x != 0) return;
    if (tid == 0) s_base = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += kDecThreads) {
      const int seq = b0 + tid;
      const long long x =
          seq < a.c.B ? (long long)visible_span(cache_len(a.c, seq), a.window, a.sinks).vb * HG : 0;
      long long v = x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = v;
      __syncthreads();
      long long before = s_base + v - x;
      for (int w = 0; w < warp; ++w) before += s_sum[w];
      if (blockIdx.x == 0 && seq < a.c.B) a.prefix[seq] = before;
      if (before <= u && u < before + x) {
        s_b = seq;
        s_off = u - before;
      }
      __syncthreads();
      if (tid == kDecThreads - 1) s_base = before + x;
    }
    __syncthreads();
    if (u >= u_end) return;
    b = s_b;
    off = s_off;
  } else {
    b = blockIdx.x / HG;
    const int n = cache_len(a.c, b);
    if (blockIdx.x % HG == 0 && tid == 0 && a.c.lens[b] != n) record_page_error();
    u = 0;
    u_end = visible_span(n, a.window, a.sinks).vb;
    off = (blockIdx.x % HG) * u_end;
    if (u_end == 0) {  // no key: o = 0
      const int gt = blockIdx.x % a.GT, nh = min(MT, a.G - gt * MT);
      const int hq0 = blockIdx.x % HG / a.GT * a.G + gt * MT;
      for (int r = warp; r < nh; r += kDecWarps) {
        for (int d = lane; d < D; d += 32) store16(a.o, ((int64_t)b * a.Hq + hq0 + r) * D + d, 0.0f, a.q_fp16);
        write_lse<D>(a, b, hq0 + r, -INFINITY, 0.0f);
      }
      return;
    }
  }

  uint8_t* ring = smem + warp * Tile::kWarpBytes;
  const uint32_t ring_u = smem_u32(ring);
  // this lane's 16 bytes of the rows of a load: offset in a page, place in the ring
  const int ld_row = lane / kChunks, ld_chunk = lane % kChunks;
  const int row_bytes = (int)(a.c.rs * E);
  const int64_t ld_off = ld_row * row_bytes + ld_chunk * 16;
  // ldmatrix: row of K (rows of a matrix are keys), row of V (transposed); the chunk's number is XORed in
  const uint32_t k_lane = swz<kRow>((lane / 16) * 8 + lane % 8, lane / 8 & 1);
  const uint32_t v_lane = swz<kRow>((lane / 8 & 1) * 8 + lane % 8, lane / 16);

  while (u < u_end) {
    const Span sp = visible_span(cache_len(a.c, b), a.window, a.sinks);
    if (SPLIT && sp.vb == 0) {  // an empty sequence between two
      ++b;
      continue;
    }
    const int row = (int)(off / sp.vb), blk0 = (int)(off % sp.vb);
    const int nblk = (int)min((long long)(sp.vb - blk0), u_end - u);
    const int h = row / a.GT, gt = row % a.GT;
    const int hq0 = h * a.G + gt * MT;
    const int nh = min(MT, a.G - gt * MT);
    const int* table = a.c.table + (int64_t)b * a.c.max_pages;

    // ---- Q fragments (A operand: rows are query heads)
    uint32_t qa[D / 16][MT == 16 ? 4 : 2];
    float qs[2] = {a.scale_log2, a.scale_log2};
#pragma unroll
    for (int half = 0; half < MT / 8; ++half) {
      const int r = lane / 4 + 8 * half;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + ((int64_t)b * a.Hq + hq0 + r) * (D / 2);
      if constexpr (CT != kQ8) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qa[k][half] = r < nh ? q[k * 8 + (lane & 3)] : 0u;
          qa[k][half + MT / 8] = r < nh ? q[k * 8 + 4 + (lane & 3)] : 0u;
        }
      } else {
        // fp16 for the exact INT8 keys: scaled by a power of two (exact) so
        // that a bf16 query fits; the lane's elements are 4 (lane % 4) + 0..3
        float f[D / 16][4];
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint2 w = r < nh ? reinterpret_cast<const uint2*>(q)[k * 4 + (lane & 3)] : make_uint2(0, 0);
          const float2 x = a.q_fp16 ? unpack2<__half>(w.x) : unpack2<__nv_bfloat16>(w.x);
          const float2 y = a.q_fp16 ? unpack2<__half>(w.y) : unpack2<__nv_bfloat16>(w.y);
          f[k][0] = x.x, f[k][1] = x.y, f[k][2] = y.x, f[k][3] = y.y;
#pragma unroll
          for (int i = 0; i < 4; ++i) amax = max_nan(amax, fabsf(f[k][i]));
        }
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int ex = (int)(__float_as_uint(amax) >> 23);
        const int e = ex == 0 || ex == 255 ? 0 : min(100, 14 - (ex - 127));
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        qs[half] = a.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const __half2 x = __floats2half2_rn(f[k][0] * up, f[k][1] * up);
          const __half2 y = __floats2half2_rn(f[k][2] * up, f[k][3] * up);
          qa[k][half] = *reinterpret_cast<const uint32_t*>(&x);
          qa[k][half + MT / 8] = *reinterpret_cast<const uint32_t*>(&y);
        }
      }
    }

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int v_exp = -100;
    float v_unit = __uint_as_float((127 + 14 + 100) << 23);  // 2^(14 - v_exp)

    const int mine_n = nblk > warp ? (nblk - warp + kDecWarps - 1) / kDecWarps : 0;
    auto page_of = [&](int i) {  // page of the warp's i-th block (0 behind the last)
      if (i >= mine_n) return 0;
      const int key = span_block(sp, blk0 + warp + i * kDecWarps) * kBlk;
      return __ldg(table + (key >> a.c.page_log2));
    };
    const uint8_t* k_base = static_cast<const uint8_t*>(a.c.k) + h * a.c.hs * E + ld_off;
    const uint8_t* v_base = static_cast<const uint8_t*>(a.c.v) + h * a.c.hs * E + ld_off;
    // whether every key of a block is visible
    auto whole_block = [&](int key) { return key + kBlk <= sp.n && (key >= sp.ws || key + kBlk <= a.sinks); };
    uint32_t okay = 0;  // bit x: the page of the block loaded x loads ago is one
    auto load = [&](int i, int pid) {
      okay <<= 1;
      if (i < mine_n) {
        const int key = span_block(sp, blk0 + warp + i * kDecWarps) * kBlk;
        const bool ok = (uint32_t)pid < (uint32_t)a.c.n_pages;
        if (!ok) {
          record_page_error();
          pid = 0;
        }
        okay |= ok;
        const uint32_t dst = ring_u + (i % S) * Tile::kStage;
        const int off0 = key & page_mask;
        const int64_t at = (int64_t)pid * (a.c.page_stride * E) + (int64_t)off0 * row_bytes;
        const uint8_t *kp = k_base + at, *vp = v_base + at;
        const uint32_t kd = dst + swz<kRow>(ld_row, ld_chunk);
        // (rows kRowsPerLoad x further down: the swizzle XORs the chunk with a function of the row)
        auto place = [&](int x) { return kd + x * 512 ^ (swz<kRow>(x * kRowsPerLoad, 0) & (kRow - 1)); };
        if (ok && whole_block(key)) {
          if (row_bytes == kRow) {  // rows next to each other: constant offsets
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
              cp_async16(place(x), kp + x * 512);
              cp_async16(place(x) + Tile::kBlkBytes, vp + x * 512);
            }
          } else {
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
              cp_async16(place(x), kp + (int64_t)(x * kRowsPerLoad) * row_bytes);
              cp_async16(place(x) + Tile::kBlkBytes, vp + (int64_t)(x * kRowsPerLoad) * row_bytes);
            }
          }
        } else {
#pragma unroll
          for (int x = 0; x < kLoads; ++x) {
            const int j = key + x * kRowsPerLoad + ld_row;
            const bool see = ok && j < sp.n && (j >= sp.ws || j < a.sinks);
            cp_async16(place(x), kp + (int64_t)(x * kRowsPerLoad) * row_bytes, see);
            cp_async16(place(x) + Tile::kBlkBytes, vp + (int64_t)(x * kRowsPerLoad) * row_bytes, see);
          }
        }
        if (CT == kQ8 && lane < 8) {
          const float* sc = (lane < 4 ? a.c.ks : a.c.vs) + ((int64_t)pid * a.c.H + h) * (page_mask + 1) + off0;
          cp_async16(dst + 2 * Tile::kBlkBytes + lane * 16, sc + (lane & 3) * 4, ok);
        }
      }
      cp_commit();
    };

    int pid_next = page_of(0);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      const int pid = pid_next;
      pid_next = page_of(i + 1);
      load(i, pid);
    }
    for (int it = 0; it < mine_n; ++it) {
      cp_wait<S - 2>();
      __syncwarp();
      {
        const int pid = pid_next;
        pid_next = page_of(it + S);
        load(it + S - 1, pid);
      }
      const uint32_t kt = ring_u + (it % S) * Tile::kStage, vt = kt + Tile::kBlkBytes;
      const float* sc = reinterpret_cast<const float*>(ring + (it % S) * Tile::kStage + 2 * Tile::kBlkBytes);
      const int ord = blk0 + warp + it * kDecWarps;
      const int key = span_block(sp, ord) * kBlk;
      const bool ok = okay >> (S - 1) & 1;
      const bool whole = ok && whole_block(key);  // else some keys are masked

      // ---- S = Q K^T: two n-tiles of 8 keys
      float s[2][4] = {};
      if constexpr (CT != kQ8) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t r[4];
          ldsm4(r, (kt + k_lane) ^ (32 * k));
          const uint32_t a1 = q_frag<MT, 1>(qa[k]), a2 = q_frag<MT, 2>(qa[k]), a3 = q_frag<MT, 3>(qa[k]);
          mma16816<CT == kBF16>(s[0], qa[k][0], a1, a2, a3, r[0], r[1]);
          mma16816<CT == kBF16>(s[1], qa[k][0], a1, a2, a3, r[2], r[3]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {
          uint32_t r[4];
          ldsm4(r, (kt + k_lane) ^ (16 * k));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a1 = q_frag<MT, 1>(qa[k + x]), a2 = q_frag<MT, 2>(qa[k + x]), a3 = q_frag<MT, 3>(qa[k + x]);
            uint32_t b0, b1;
            int8x4_to_half(r[x], b0, b1);
            mma16816<false>(s[0], qa[k + x][0], a1, a2, a3, b0, b1);
            int8x4_to_half(r[2 + x], b0, b1);
            mma16816<false>(s[1], qa[k + x][0], a1, a2, a3, b0, b1);
          }
        }
      }
      // ---- scale, mask; s[t][c]: head lane / 4 (+ 8), key 8 t + 2 (lane % 4) + (c & 1)
      float vs[2][2];
      if constexpr (CT == kQ8) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float2 ks = *reinterpret_cast<const float2*>(sc + 8 * t + 2 * (lane & 3));
          const float2 v2 = *reinterpret_cast<const float2*>(sc + 16 + 8 * t + 2 * (lane & 3));
          vs[t][0] = v2.x;
          vs[t][1] = v2.y;
#pragma unroll
          for (int c = 0; c < 4; ++c) s[t][c] *= (c & 1) ? ks.y : ks.x;
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < MT / 4; ++c) s[t][c] *= qs[c >> 1];
      if (!whole) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int j = key + 8 * t + 2 * (lane & 3) + c;
            if (!(ok && j < sp.n && (j >= sp.ws || j < a.sinks))) {
              s[t][c] = s[t][2 + c] = -INFINITY;
              if (CT == kQ8) vs[t][c] = 0.0f;
            }
          }
      }
      if constexpr (CT == kQ8) {
        // the weights times V's scales are held as fp16 in units of 2^(v_exp - 14), v_exp above every scale so far
        const float top = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]));
        if (__any_sync(0xffffffffu, top * v_unit >= 16384.0f)) {
          float x = top;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          const int e = (int)(__float_as_uint(x) >> 23) - 126;  // x < 2^e (x is above 2^-101)
          if (e <= 128) {
            const float down = __uint_as_float((uint32_t)max(127 + v_exp - e, 0) << 23);
            v_exp = e;
            v_unit = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) o[n][c] *= down;
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) vs[t][c] *= v_unit;
      }
      // ---- online softmax
      float p[2][4];
#pragma unroll
      for (int half = 0; half < MT / 8; ++half) {
        float mx = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mx = fmaxf(mx, s[t][2 * half + c]);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[half], mx), ms = mn == -INFINITY ? 0.0f : mn;
        const float alpha = exp2f(m[half] - ms);
        m[half] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float e = exp2f(s[t][2 * half + c] - ms);
            p[t][2 * half + c] = e;
            sum += e;
          }
        l[half] = l[half] * alpha + sum;
        if (__any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[n][2 * half] *= alpha;
            o[n][2 * half + 1] *= alpha;
            if (MT == 8) {
              o[n][2] *= alpha;
              o[n][3] *= alpha;
            }
          }
        }
        if (a.scores) {
          const int r = lane / 4 + 8 * half;
          if (r < nh) {
            float* dst = a.scores + ((int64_t)b * a.Hq + hq0 + r) * a.score_cap + (int64_t)ord * kBlk + 2 * (lane & 3);
#pragma unroll
            for (int t = 0; t < 2; ++t)
              *reinterpret_cast<float2*>(dst + 8 * t) = make_float2(s[t][2 * half], s[t][2 * half + 1]);
          }
        }
      }
      // ---- O += P V, the weights as hi + lo
      uint32_t hi[4], lo[4];  // fragment order: (head, keys 0-7), (head + 8, keys 0-7), (head, 8-15), (head + 8, 8-15)
#pragma unroll
      for (int half = 0; half < MT / 8; ++half)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float x = p[t][2 * half], y = p[t][2 * half + 1];
          if constexpr (CT == kQ8) {
            x *= vs[t][0];
            y *= vs[t][1];
          } else {
            x *= kUnit;
            y *= kUnit;
          }
          split_pair<kVB>(x, y, hi[2 * t + half], lo[2 * t + half]);
        }
      if constexpr (MT == 8) {
        hi[1] = lo[0];
        hi[3] = lo[2];
      }
      if constexpr (CT != kQ8) {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t r[4];
          ldsm4t(r, (vt + v_lane) ^ (16 * n));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mma16816<kVB>(o[n + x], hi[0], hi[1], hi[2], hi[3], r[2 * x], r[2 * x + 1]);
            if (MT == 16) mma16816<kVB>(o[n + x], lo[0], lo[1], lo[2], lo[3], r[2 * x], r[2 * x + 1]);
          }
        }
      } else {
        // chunk c holds channels 16 c + 0..15; a transposed 16-bit load gives
        // the channel pair 16 c + 2 n, + 1 of two keys: o[2 c] takes the even
        // channels, o[2 c + 1] the odd ones
#pragma unroll
        for (int c = 0; c < NT / 2; c += 2) {
          uint32_t r[4];
          ldsm4t(r, (vt + v_lane) ^ (16 * c));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t e0, o0, e1, o1;
            e4m3x4_to_half(r[2 * x], e0, o0);
            e4m3x4_to_half(r[2 * x + 1], e1, o1);
            float(&oe)[4] = o[2 * (c + x)];
            float(&oo)[4] = o[2 * (c + x) + 1];
            mma16816<kVB>(oe, hi[0], hi[1], hi[2], hi[3], e0, e1);
            mma16816<kVB>(oo, hi[0], hi[1], hi[2], hi[3], o0, o1);
            if (MT == 16) {
              mma16816<kVB>(oe, lo[0], lo[1], lo[2], lo[3], e0, e1);
              mma16816<kVB>(oo, lo[0], lo[1], lo[2], lo[3], o0, o1);
            }
          }
        }
      }
      __syncwarp();  // the ring slot may be filled again
    }
    cp_wait<0>();
    __syncthreads();  // every warp is done with its ring: the merge uses it

    // ---- merge the warps
    float* so = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int half = 0; half < MT / 8; ++half) {
      float x = l[half];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      const int r = lane / 4 + 8 * half;
      if ((lane & 3) == 0) {
        s_m[warp][r] = m[half];
        s_l[warp][r] = x;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x0 = o[n][2 * half], x1 = o[n][2 * half + 1];
        if (MT == 8) {
          x0 += o[n][2];
          x1 += o[n][3];
        }
        if constexpr (CT == kQ8) {
          x0 *= __uint_as_float((uint32_t)(127 - 14 + v_exp) << 23);
          x1 *= __uint_as_float((uint32_t)(127 - 14 + v_exp) << 23);
        } else {
          x0 *= 1.0f / kUnit;
          x1 *= 1.0f / kUnit;
        }
        if constexpr (CT != kQ8) {
          so[r * D + n * 8 + 2 * (lane & 3)] = x0;
          so[r * D + n * 8 + 2 * (lane & 3) + 1] = x1;
        } else {  // columns 2 (lane % 4) + 0, 1 of the even or odd channels
          so[r * D + (n / 2) * 16 + 4 * (lane & 3) + (n & 1)] = x0;
          so[r * D + (n / 2) * 16 + 4 * (lane & 3) + 2 + (n & 1)] = x1;
        }
      }
    }
    __syncthreads();
    const bool alone = !SPLIT || (blk0 == 0 && nblk == sp.vb);
    const int slot = 2 * blockIdx.x + (first_piece ? 0 : 1);
    for (int r = warp; r < nh; r += kDecWarps) {
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, s_m[w][r]);
      const float ms = mm == -INFINITY ? 0.0f : mm;
      float ll = 0.0f, f[kDecWarps];
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        f[w] = exp2f(s_m[w][r] - ms);
        ll += s_l[w][r] * f[w];
      }
      const float inv = alone ? (ll > 0.0f || isnan(ll) ? 1.0f / ll : 0.0f) : 1.0f;
      for (int d = lane; d < D; d += 32) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w)
          x += reinterpret_cast<const float*>(smem + w * Tile::kWarpBytes)[r * D + d] * f[w];
        if (alone) store16(a.o, ((int64_t)b * a.Hq + hq0 + r) * D + d, x * inv, a.q_fp16);
        else a.part_o[((int64_t)slot * kMaxGroup + r) * D + d] = x;
      }
      if (alone) {
        write_lse<D>(a, b, hq0 + r, mm, ll);
        if (!SPLIT && lane == 0) s_lse[r] = ll > 0.0f || isnan(ll) ? mm + log2f(ll) : -INFINITY;
      } else if (lane == 0) {
        a.part_m[slot * kMaxGroup + r] = mm;
        a.part_l[slot * kMaxGroup + r] = ll;
      }
    }
    __syncthreads();  // the rings may be filled again
    if (!SPLIT && a.scores && a.GT == 1) {  // (more tiles of a group share the weights: decode_weight_kernel)
      add_weights(a, sp, b, h, tid, kDecThreads, [&](int g) { return s_lse[g]; });
    }
    u += nblk;
    off += nblk;
    first_piece = false;
    if (off == (long long)sp.vb * HG) {
      off = 0;
      ++b;
    }
  }
}

// Joins the pieces of a row in the order of their CTAs; one CTA a (sequence,
// query head).  Rows that one CTA did alone are done already.  A few long rows
// have a piece for every CTA of the split, which 512 threads read four (D = 128)
// at a time: 64 us against 72 with 128 threads for 32 heads over 131k tokens.
// Many rows have a piece or two each: 284 us with 128 threads against 299 for
// 64 x 64 heads.
template <int D, int MT, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const DecodeArgs a) {
  __shared__ float s_f[kDecodeCtas];
  __shared__ float s_x[kJoinThreads], s_w[kJoinThreads / 32];
  pdl_launch();
  pdl_wait();
  const int tid = threadIdx.x;
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq;
  const int h = hq / a.G, g = hq % a.G, r = g % MT;
  const int vb = visible_span(cache_len(a.c, b), a.window, a.sinks).vb;
  const int64_t out = ((int64_t)b * a.Hq + hq) * D;
  if (vb == 0) {
    if (tid < D) store16(a.o, out + tid, 0.0f, a.q_fp16);
    if (tid < 32) write_lse<D>(a, b, hq, -INFINITY, 0.0f);
    return;
  }
  const long long share = a.prefix[a.c.B];
  const long long u = a.prefix[b] + (long long)(h * a.GT + g / MT) * vb;
  const int c0 = (int)(u / share), c1 = (int)((u + vb - 1) / share), n = c1 - c0 + 1;
  if (n == 1) return;
  auto slot = [&](int i) { return 2 * (c0 + i) + (i == 0 && u != c0 * share ? 1 : 0); };
  // of x over the CTA: sum or maximum
  auto all = [&](float x, auto f) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, d));
    __syncthreads();
    if ((tid & 31) == 0) s_w[tid >> 5] = x;
    __syncthreads();
    x = s_w[0];
#pragma unroll
    for (int w = 1; w < kJoinThreads / 32; ++w) x = f(x, s_w[w]);
    return x;
  };
  // largest m, factors of the pieces, l
  float mx = -INFINITY;
  for (int i = tid; i < n; i += kJoinThreads) mx = fmaxf(mx, a.part_m[slot(i) * kMaxGroup + r]);
  mx = all(mx, [](float x, float y) { return fmaxf(x, y); });
  const float ms = mx == -INFINITY ? 0.0f : mx;
  float l = 0.0f;
  for (int i = tid; i < n; i += kJoinThreads) {
    const float f = exp2f(a.part_m[slot(i) * kMaxGroup + r] - ms);
    s_f[i] = f;
    l += f * a.part_l[slot(i) * kMaxGroup + r];
  }
  l = all(l, [](float x, float y) { return x + y; });
  constexpr int P = kJoinThreads / D;  // pieces summed side by side
  const int d = tid % D;
  float x = 0.0f;
#pragma unroll 8
  for (int i = tid / D; i < n; i += P) x += s_f[i] * a.part_o[((int64_t)slot(i) * kMaxGroup + r) * D + d];
  s_x[tid] = x;
  __syncthreads();
  if (tid < D) {
#pragma unroll
    for (int p = 1; p < P; ++p) x += s_x[tid + p * D];
    store16(a.o, out + d, l > 0.0f || isnan(l) ? x / l : 0.0f, a.q_fp16);
  }
  if (tid < 32) write_lse<D>(a, b, hq, mx, l);
}

// the weights of all keys
__global__ void __launch_bounds__(256) decode_weight_kernel(const DecodeArgs a) {
  pdl_wait();
  const int b = blockIdx.x / a.c.H, h = blockIdx.x % a.c.H;
  const Span sp = visible_span(cache_len(a.c, b), a.window, a.sinks);
  const float* lse2 = a.lse2 + (int64_t)b * a.Hq + h * a.G;
  add_weights(a, sp, b, h, blockIdx.y * 256 + threadIdx.x, gridDim.y * 256, [&](int g) { return lse2[g]; });
}

template <int D, int CT, int MT>
cudaError_t launch_decode_t(const DecodeArgs& a, cudaStream_t st) {
  constexpr int smem = kDecWarps * DecTile<D, CT>::kWarpBytes;
  static_assert(MT * D * 4 <= DecTile<D, CT>::kWarpBytes, "a warp's ring holds its rows of O for the merge");
  const int64_t want = (a.score_cap + 1023) / 1024;  // four keys a thread
  const dim3 weights((unsigned)(a.c.B * a.c.H), (unsigned)(want < 64 ? want : 64));
  cudaError_t e;
  if (a.direct) {
    auto kernel = decode_kernel<D, CT, MT, false>;
    static DeviceOnce once;
    e = once.run([&](int) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(a.c.B * a.c.H * a.GT), kDecThreads, smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess || !a.scores || a.GT == 1) return e;
    decode_weight_kernel<<<weights, 256, 0, st>>>(a);
    return cudaGetLastError();
  }
  auto kernel = decode_kernel<D, CT, MT, true>;
  static DeviceOnce once;
  int wave = 0;  // CTAs that run at a time
  e = once.run([&](int dev) {
    int sms = 0, per = 0;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kDecThreads, smem);
    once.value[dev] = sms * (per < 1 ? 1 : per);
    return e;
  }, &wave);
  if (e != cudaSuccess) return e;
  // one wave; no more CTAs than the smallest shares of the longest sequences
  const int64_t blocks = (int64_t)a.c.B * a.c.H * a.GT * ((a.c.cap + kBlk - 1) / kBlk);
  int64_t ctas = (blocks + kMinShare - 1) / kMinShare;
  if (ctas > wave) ctas = wave;
  if (ctas > kDecodeCtas) ctas = kDecodeCtas;
  kernel<<<(unsigned)ctas, kDecThreads, smem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t heads = (int64_t)a.c.B * a.Hq;
  e = heads <= 296 ? launch_pdl(decode_join_kernel<D, MT, 512>, dim3((unsigned)heads), dim3(512), 0, st, a)
                   : launch_pdl(decode_join_kernel<D, MT, 128>, dim3((unsigned)heads), dim3(128), 0, st, a);
  if (e != cudaSuccess || !a.scores) return e;
  return launch_pdl(decode_weight_kernel, weights, dim3(256), 0, st, a);
}

template <int D, int CT>
cudaError_t launch_decode_m(const DecodeArgs& a, cudaStream_t st) {
  return a.G <= 8 ? launch_decode_t<D, CT, 8>(a, st) : launch_decode_t<D, CT, 16>(a, st);
}
template <int D>
cudaError_t launch_decode_d(const DecodeArgs& a, int quantized, cudaStream_t st) {
  if (quantized) return launch_decode_m<D, kQ8>(a, st);
  return a.q_fp16 ? launch_decode_m<D, kFP16>(a, st) : launch_decode_m<D, kBF16>(a, st);
}

}  // namespace

cudaError_t launch_attn_decode(const DecodeArgs& a, int quantized, cudaStream_t st) {
  return a.c.D == 128 ? launch_decode_d<128>(a, quantized, st) : launch_decode_d<64>(a, quantized, st);
}

}  // namespace sage
