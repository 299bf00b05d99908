// attn_window.cu -- sliding-window attention with sinks (16-bit, forward) on the
// 5th-generation tensor core (tcgen05), accumulators in TMEM.
//
// For query row p of a head, over the visible keys j (j <= p and (p - j < window
// or j < sinks)):  S_j = q . K_j,  o = sum_j e^(sm_scale (S_j - m)) V_j / l,
// l = sum_j e^(sm_scale (S_j - m)),  lse = sm_scale m + ln l.  One pass: m and l
// run along the key tiles.  m is the row's maximum only to within a factor 2^8
// of the weights: as long as no score lies more than 8 (in base 2) above it, O
// needs no rescaling, and m cancels in o and lse whatever it is.
//
// A work item is 256 query rows of one head: two tiles of 128 rows that share
// every 128-key tile of K and V.  One CTA an SM takes items in turn (persistent:
// the next item's loads and first products run under the last one's softmax and
// output).  512 threads in four warpgroups:
//   WG0, 1  softmax of row tile 0 and 1 (thread = row = TMEM lane)
//   WG2     output of both tiles
//   WG3     warp 0: TMA producer; warp 1: MMA issuer (one thread) and TMEM owner
// TMEM (512 columns): S_i at 128 i; P_i (16 bit) over the upper half of S_i, as
// the A operand of P V; O_i at 256 + D i.  A row tile's chain is
// S(0) P V(0) S(1) ...; the two tiles' chains keep the tensor core busy while
// the other tile's softmax runs.
//
// Keys a row does not see are -inf before the maximum, so their weights are
// exact zeros; a NaN or infinity in such a key's V still makes 0 x inf = NaN in
// the product, so a row whose output is not finite is computed again over its
// visible keys alone (window_row).  Rows of V behind a sequence's end (padding,
// which may hold anything) are zeroed in shared memory first.
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "serving.cuh"

namespace sage {

namespace {

constexpr int kWinThreads = 512;
constexpr int kNarrow = 32;            // rows of the narrow key tile (few sinks)
constexpr float kWinSlack = 8.0f;      // log2 of the largest weight before O is rescaled
// registers a thread of the softmax, output and producer / MMA warpgroups
constexpr uint32_t kWinRegsSoftmax = 192, kWinRegsOut = 80, kWinRegsIssue = 48;
static_assert(2 * kWinRegsSoftmax + kWinRegsOut + kWinRegsIssue <= 512, "register split exceeds the launch");

template <int D>
struct WinSmem {
  static constexpr uint32_t kTileBytes = 128 * D * 2;
  static constexpr int kRing = D == 128 ? 5 : 8;  // K and V tiles in turn
  static constexpr uint32_t oRing = 2 * kTileBytes;
  static constexpr uint32_t oL = oRing + kRing * kTileBytes;  // float2[2][128]: l, sm_scale log2(e) m
  static constexpr uint32_t oBar = oL + 2 * 128 * 8;
  static constexpr uint32_t kBars = 2 * kRing + 1 + 2 * 9 + 1;
  static constexpr uint32_t oTmem = oBar + 8 * kBars;
  static constexpr uint32_t kBytes = oTmem + 16;
  static_assert(kBytes <= 227 * 1024, "window attention buffers exceed the shared memory of one CTA");
};

// The key tiles of a work item: sink tiles [0, ns) with keys 128 j.., then the
// tiles of the window, keys 128 (t0 + j - ns)..  Row tile i takes the sink tiles
// and [lo[i], hi[i]].
struct WinItem {
  int b, h, q0, n;
  int ns, t0, nt;
  int lo[2], hi[2];
  __device__ __forceinline__ int count(int i) const { return hi[i] < lo[i] ? 0 : ns + hi[i] - lo[i] + 1; }
  __device__ __forceinline__ int tile(int i, int k) const { return k < ns ? k : lo[i] + k - ns; }
  __device__ __forceinline__ int key0(int j) const { return 128 * (j < ns ? j : t0 + j - ns); }
};

__device__ __forceinline__ WinItem win_item(const WindowArgs& a, int idx) {
  // heads in groups whose K and V stay in L2 while every pair of their rows runs, heaviest rows first
  WinItem w;
  const int pairs = (a.N + 255) / 256, per = a.group * pairs;
  const int g = idx / per, in = idx % per;
  const int heads = min(a.group, a.B * a.Hq - g * a.group);
  const int bh = g * a.group + in % heads;
  w.b = bh / a.Hq;
  w.h = bh % a.Hq;
  w.q0 = 256 * (pairs - 1 - in / heads);
  w.n = a.lens ? min(max(__ldg(a.lens + w.b), 0), a.N) : a.N;
  int first[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int lead = w.q0 + 128 * i - a.window + 1;
    first[i] = a.window > 0 && lead > 0 ? lead / 128 : 0;
  }
  if (a.sinks > 128 * first[0]) first[0] = first[1] = 0;  // the sinks reach into the window's tiles
  w.t0 = first[0];
  w.ns = w.t0 > 0 ? (a.sinks + 127) / 128 : 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w.lo[i] = w.ns + first[i] - w.t0;
    w.hi[i] = w.q0 + 128 * i < w.n ? w.ns + w.q0 / 128 + i - w.t0 : w.lo[i] - 1;
  }
  w.nt = w.count(0) == 0 ? 0 : max(w.hi[0], w.hi[1]) + 1;
  return w;
}
__device__ __forceinline__ bool win_narrow(const WindowArgs& a, const WinItem& w, int j) {
  return j == w.ns - 1 && a.sinks - 128 * j <= kNarrow;
}

// One row by one warp, over its visible keys alone: lane = key for the scores,
// lane = D / 32 channels for P V.
template <typename T, int D>
__device__ __forceinline__ void window_row(const WindowArgs& a, int b, int hq, int i) {
  const int lane = threadIdx.x & 31;
  const int hk = hq / (a.Hq / a.Hkv);
  const int64_t qrow = row_offset((int64_t)b * a.Hq + hq, i, a.Hq, a.N, D, a.nhd);
  const int64_t krow = row_offset((int64_t)b * a.Hkv + hk, 0, a.Hkv, a.N, D, a.nhd);
  const int64_t ks = row_stride(a.Hkv, D, a.nhd);
  const T* k = static_cast<const T*>(a.k) + krow;
  const T* v = static_cast<const T*>(a.v) + krow;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + qrow);
  const int ws = a.window > 0 && i + 1 > a.window ? i + 1 - a.window : 0;
  float m = -INFINITY, l = 0.0f, o[D / 32] = {};
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int lo = part == 0 ? 0 : ws, hi = part == 0 ? min(a.sinks, ws) : i + 1;
#pragma unroll 1
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      float t = -INFINITY;
      if (j < hi) {
        const uint4* row = reinterpret_cast<const uint4*>(k + j * ks);
        float x = 0.0f;
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = row[c], y = q[c];
          const uint32_t u[4] = {w.x, w.y, w.z, w.w}, z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<T>(u[e]), g = unpack2<T>(z[e]);
            x = fmaf(f.x, g.x, x);
            x = fmaf(f.y, g.y, x);
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
#pragma unroll 1
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
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// the low n bits (n taken as the nearest of 0 and 32)
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

__device__ __forceinline__ void store_row32(void* p, const uint32_t* w, bool wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

struct WinBars {
  uint64_t* kv_full;   // [ring]
  uint64_t* kv_empty;  // [ring]  both row tiles' products that read the slot retired
  uint64_t* part;      // a tile of V that ends behind the sequence landed (its producer zeroes those rows)
  uint64_t* q_full;    // [2]
  uint64_t* q_empty;   // [2]  the item's last Q K^T of tile i retired
  uint64_t* s_full;    // [2]  Q K^T of tile i retired
  uint64_t* p_full;    // [2]  P_i written (one arrival a warp)
  uint64_t* o_done;    // [2]  a P V of tile i retired
  uint64_t* o_full;    // [2]  the item's last P V of tile i retired
  uint64_t* o_free;    // [2]  the item's O_i, l and m have been read (one arrival a warp)
  uint64_t* l_ready;   // [2]  l and m of tile i in shared memory (one arrival a warp)
  uint64_t* mma_done;  // all tensor-core work of the CTA retired
};

template <typename T, int D>
__global__ void __launch_bounds__(kWinThreads, 1)
    attn_window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKn,
                       const __grid_constant__ CUtensorMap tmVn, const __grid_constant__ WindowArgs a) {
  using L = WinSmem<D>;
  constexpr int R = L::kRing;
  constexpr uint32_t kF16 = std::is_same<T, __half>::value ? 0u : 1u;  // operand format: fp16 or bf16
  constexpr uint32_t kTransB = 1u << 16;                               // B with its N dimension contiguous
  constexpr uint32_t kIdescQK = make_idesc(1, kF16, kF16, 128, 128), kIdescQKn = make_idesc(1, kF16, kF16, 128, kNarrow);
  constexpr uint32_t kIdescPV = make_idesc(1, kF16, kF16, 128, D) | kTransB;
  constexpr uint32_t kTmemCols = 512, kP = 64;  // kP: P_i's first column in S_i

  extern __shared__ __align__(1024) uint8_t smem_win[];
  uint8_t* sQ = smem_win;
  uint8_t* ring = smem_win + L::oRing;
  float2* s_l = reinterpret_cast<float2*>(smem_win + L::oL);
  WinBars bar;
  bar.kv_full = reinterpret_cast<uint64_t*>(smem_win + L::oBar);
  bar.kv_empty = bar.kv_full + R;
  bar.part = bar.kv_empty + R;
  bar.q_full = bar.part + 1;
  bar.q_empty = bar.q_full + 2;
  bar.s_full = bar.q_empty + 2;
  bar.p_full = bar.s_full + 2;
  bar.o_done = bar.p_full + 2;
  bar.o_full = bar.o_done + 2;
  bar.o_free = bar.o_full + 2;
  bar.l_ready = bar.o_free + 2;
  bar.mma_done = bar.l_ready + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_win + L::oTmem);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, wg = warp / 4;
  if (threadIdx.x == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(&bar.kv_full[s], 1);
      mbar_init(&bar.kv_empty[s], 1);
    }
    mbar_init(bar.part, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.o_done[i], 1);
      mbar_init(&bar.o_full[i], 1);
      mbar_init(&bar.o_free[i], 4);
      mbar_init(&bar.l_ready[i], 4);
    }
    mbar_init(bar.mma_done, 1);
    mbar_fence_init();
  }
  if (warp == 13) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (wg == 3) {
    regs_dec<kWinRegsIssue>();
    if (warp == 12) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
      }
      bool ok = true;
      uint32_t idx = 0, parts = 0;  // ring slots filled, partial tiles of V
      uint32_t nq[2] = {0, 0};      // items of tile i
      const int G = a.Hq / a.Hkv;
      for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
        const WinItem w = win_item(a, it);
        const int hk = w.h / G;
        for (int j = 0; j < w.nt && ok; ++j) {
          const bool narrow = win_narrow(a, w, j);
          const int key0 = w.key0(j);
          const uint32_t rows = narrow ? kNarrow : 128, bytes = rows * D * 2, half = rows * 128;
          for (int x = 0; x < 2 && ok; ++x, ++idx) {  // K, then V
            const uint32_t s = idx % R;
            // rows of V from here on belong to no token of this sequence (TMA zeroes those behind N itself)
            const bool part = x == 1 && w.n < a.N && key0 + (int)rows > w.n;
            uint8_t* dst = ring + s * L::kTileBytes;
            uint64_t* full = part ? bar.part : &bar.kv_full[s];
            if (lane == 0) {
              ok = mbar_wait(&bar.kv_empty[s], ((idx / R) + 1) & 1);
              if (ok) {
                mbar_expect_tx(full, bytes);
                const CUtensorMap* m = x == 0 ? (narrow ? &tmKn : &tmK) : (narrow ? &tmVn : &tmV);
                for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * half, m, full, 64 * c, key0, hk, w.b);
                if (part) ok = mbar_wait(full, parts & 1);
              }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            if (part && ok) {
              ++parts;
              for (int r = w.n - key0; r < (int)rows; ++r)
                for (int c = lane; c < D / 8; c += 32)
                  *reinterpret_cast<uint4*>(dst + (c / 8) * half + r * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.kv_full[s]);
            }
            if (j == 0 && x == 0 && ok && lane == 0) {
              // Q after the first K: it waits for the last item's last product
              for (int i = 0; i < 2; ++i) {
                if (w.count(i) == 0) continue;
                if (nq[i] > 0 && !(ok = mbar_wait(&bar.q_empty[i], (nq[i] - 1) & 1))) break;
                mbar_expect_tx(&bar.q_full[i], L::kTileBytes);
                for (int c = 0; c < D / 64; ++c)
                  tma_load_4d(sQ + i * L::kTileBytes + c * 128 * 128, &tmQ, &bar.q_full[i], 64 * c, w.q0 + 128 * i,
                              w.h, w.b);
                ++nq[i];
              }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
          }
        }
      }
      // never leave a copy in flight
      if (lane == 0) {
        for (uint32_t x = idx > R ? idx - R : 0; x < idx; ++x) mbar_wait(&bar.kv_full[x % R], (x / R) & 1);
        for (int i = 0; i < 2; ++i)
          if (nq[i] > 0) mbar_wait(&bar.q_full[i], (nq[i] - 1) & 1);
      }
    } else if (warp == 13) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        // One chain a row tile: S(0), P V(0), S(1), ..., item after item; each step is
        // issued as soon as its operands are there (non-blocking polls).
        struct {
          WinItem w;
          int it;         // item
          int k;          // step within the item
          int g;          // key tiles of the items before this one
          uint32_t step;  // steps so far (all items)
          uint32_t items; // items before this one
          bool pv;        // the step's S is issued, its P V is not
          bool live;
        } c[2];
        auto next_item = [&](auto& ch, int i) {  // the next item that has rows in tile i
          while (ch.it < a.items) {
            ch.w = win_item(a, ch.it);
            if (ch.w.count(i) > 0) break;
            ch.g += ch.w.nt;
            ch.it += gridDim.x;
          }
          ch.live = ch.it < a.items;
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          c[i].it = blockIdx.x;
          c[i].k = c[i].g = 0;
          c[i].step = c[i].items = 0;
          c[i].pv = false;
          next_item(c[i], i);
        }
        int rel_k = 0, rel_v = 0;  // key tiles whose K, V slots are released
        bool ok = true;
        uint64_t t_idle = 0;
        while (ok && (c[0].live || c[1].live)) {
          bool progress = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            auto& ch = c[i];
            if (!ch.live) continue;
            const int j = ch.w.tile(i, ch.k);
            const uint32_t g = ch.g + j;
            const bool narrow = win_narrow(a, ch.w, j);
            if (!ch.pv) {
              const uint32_t s = (2 * g) % R;
              if ((ch.k > 0 || mbar_test_wait(smem_u32(&bar.q_full[i]), ch.items & 1)) &&
                  mbar_test_wait(smem_u32(&bar.kv_full[s]), (2 * g / R) & 1)) {
                tc_fence_after();
                const uint32_t q = smem_u32(sQ + i * L::kTileBytes), k = smem_u32(ring + s * L::kTileBytes);
                const uint32_t khalf = (narrow ? kNarrow : 128) * 128;
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                  mma_f16(tmem + 128 * i, make_sdesc(q + (x / 4) * 16384 + (x % 4) * 32, 1024, kSwizzle128B),
                          make_sdesc(k + (x / 4) * khalf + (x % 4) * 32, 1024, kSwizzle128B),
                          narrow ? kIdescQKn : kIdescQK, x > 0);
                mma_commit(&bar.s_full[i]);
                if (ch.k + 1 == ch.w.count(i)) mma_commit(&bar.q_empty[i]);
                ch.pv = true;
                progress = true;
              }
            } else {
              const uint32_t s = (2 * g + 1) % R;
              if (mbar_test_wait(smem_u32(&bar.p_full[i]), ch.step & 1) &&
                  mbar_test_wait(smem_u32(&bar.kv_full[s]), ((2 * g + 1) / R) & 1) &&
                  (ch.k > 0 || ch.items == 0 || mbar_test_wait(smem_u32(&bar.o_free[i]), (ch.items - 1) & 1))) {
                tc_fence_after();
                const uint32_t v = smem_u32(ring + s * L::kTileBytes), vhalf = (narrow ? kNarrow : 128) * 128;
                const int nk = narrow ? kNarrow / 16 : 8;
                for (int x = 0; x < nk; ++x)  // 16 keys: 8 columns of P, 16 rows of V
                  mma_f16_ts(tmem + 256 + D * i, tmem + 128 * i + kP + 8 * x,
                             make_sdesc_mn(v + x * 2048, vhalf, 1024, kSwizzle128B), kIdescPV, ch.k > 0 || x > 0);
                mma_commit(&bar.o_done[i]);
                ch.pv = false;
                ++ch.step;
                if (++ch.k == ch.w.count(i)) {
                  mma_commit(&bar.o_full[i]);
                  ch.g += ch.w.nt;
                  ch.it += gridDim.x;
                  ch.k = 0;
                  ++ch.items;
                  next_item(ch, i);
                }
                progress = true;
              }
            }
          }
          if (progress) {
            // slots that neither chain will read again
            int need_k = INT_MAX, need_v = INT_MAX;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (c[i].live) {
                const int at = c[i].g + c[i].w.tile(i, c[i].k);
                need_v = min(need_v, at);
                const int nxt = !c[i].pv ? at
                                : c[i].k + 1 < c[i].w.count(i) ? c[i].g + c[i].w.tile(i, c[i].k + 1)
                                                               : c[i].g + c[i].w.nt;
                need_k = min(need_k, nxt);
              }
            if (c[0].live || c[1].live) {
              for (; rel_k < need_k; ++rel_k) mma_commit(&bar.kv_empty[(2 * rel_k) % R]);
              for (; rel_v < need_v; ++rel_v) mma_commit(&bar.kv_empty[(2 * rel_v + 1) % R]);
            }
            t_idle = 0;
          } else if (t_idle == 0) {
            t_idle = globaltimer_ns();
          } else if (globaltimer_ns() - t_idle > g_wait_limit_ns) {
            record_error(kDevErrTimeout);
            ok = false;
          }
        }
        // every tensor-core op retired before TMEM is released
        mma_commit(bar.mma_done);
        mbar_wait(bar.mma_done, 0);
      }
      __syncwarp();
    }
  } else if (wg < 2) {
    // ------------------------------------------------------------ softmax
    regs_inc<kWinRegsSoftmax>();
    const int ti = wg, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + 128 * ti + lanes, tO = tmem + 256 + D * ti + lanes;
    const float scale = a.scale_log2, slack = kWinSlack / scale;
    uint32_t step = 0, items = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const WinItem w = win_item(a, it);
      const int count = w.count(ti);
      if (count == 0) continue;
      const int p0 = w.q0 + 128 * ti, p = p0 + row;
      float m = -INFINITY, l = 0.0f;
      for (int k = 0; k < count && ok; ++k, ++step) {
        const int j = w.tile(ti, k), key0 = w.key0(j);
        const int hi = p - key0, lo = a.window > 0 ? hi - a.window + 1 : INT_MIN, sk = a.sinks - key0;
        // columns c <= hi and (c >= lo or c < sk) are visible
        const bool masked = key0 + 127 > p0 || (a.window > 0 && p0 + 128 - a.window > key0 && sk < 128);
        const bool narrow = win_narrow(a, w, j);
        if (!(ok = mbar_wait_warp(&bar.s_full[ti], step & 1))) break;
        tc_fence_after();
        uint32_t s[128];
        tmem_ld32p(tS, s);
        if (!narrow) {
          tmem_ld32p(tS + 32, s + 32);
          tmem_ld32p(tS + 64, s + 64);
          tmem_ld32p(tS + 96, s + 96);
        }
        tmem_ld_wait();
        if (narrow) {
#pragma unroll
          for (int c = 32; c < 128; ++c) s[c] = __float_as_uint(-INFINITY);
        }
        if (masked) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t see =
                low_bits(hi + 1 - 32 * x) & (~low_bits(lo - 32 * x) | low_bits(sk - 32 * x));
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((see >> c) & 1)) s[32 * x + c] = __float_as_uint(-INFINITY);
          }
        }
        float mx8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mx8[c] = __uint_as_float(s[c]);
#pragma unroll
        for (int c = 8; c < 128; c += 16)
#pragma unroll
          for (int x = 0; x < 8; ++x)
            mx8[x] = c + 8 < 128 ? fmax3(mx8[x], __uint_as_float(s[c + x]), __uint_as_float(s[(c + 8 + x) & 127]))
                                 : fmaxf(mx8[x], __uint_as_float(s[c + x]));
        const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], fmax3(mx8[5], mx8[6], mx8[7])));
        if (m == -INFINITY) m = mx;  // nothing visible before: l = 0 and O = 0 (or unset)
        const bool grow = mx > m + slack;
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2_approx((m - mx) * scale) : 1.0f;
          if (grow) m = mx;
          l *= alpha;
          if (!(ok = mbar_wait_warp(&bar.o_done[ti], (step - 1) & 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t x[16];
            tmem_ld16p(tO + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
            tmem_st16p(tO + c, x);
          }
        }
        const float ms = m == -INFINITY ? 0.0f : m * scale;
        const float2 sc = make_float2(scale, scale), off = make_float2(-ms, -ms);
        float2 sum[4] = {};
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          if (c > 0 && narrow) break;
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 u =
                ffma2(make_float2(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1])), sc, off);
            const float2 f = make_float2(ex2_approx(u.x), ex2_approx(u.y));
            sum[(e / 2) & 3] = fadd2(sum[(e / 2) & 3], f);
            y[e / 2] = pack16<T>(f.x, f.y);
          }
          tmem_st16p(tS + kP + c / 2, y);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[ti]);
        const float2 t = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
        l += t.x + t.y;
      }
      if (!ok) break;
      // l and m for the output warps, once they have read the last item's
      if (items > 0 && !(ok = mbar_wait_warp(&bar.o_free[ti], (items - 1) & 1))) break;
      s_l[128 * ti + row] = make_float2(l, m * scale);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.l_ready[ti]);
      ++items;
    }
  } else {
    // ------------------------------------------------------------ output
    regs_dec<kWinRegsOut>();
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const bool wide = (reinterpret_cast<uintptr_t>(a.o) & 31) == 0;
    uint32_t items[2] = {0, 0};
    bool ok = true;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const WinItem w = win_item(a, it);
      for (int i = 0; i < 2 && ok; ++i) {
        if (w.count(i) == 0) continue;
        if (!(ok = mbar_wait_warp(&bar.l_ready[i], items[i] & 1))) break;
        if (!(ok = mbar_wait_warp(&bar.o_full[i], items[i] & 1))) break;
        tc_fence_after();
        ++items[i];
        const float2 lm = s_l[128 * i + row];
        const int p = w.q0 + 128 * i + row;
        const float inv = 1.0f / lm.x;
        const int64_t head = (int64_t)w.b * a.Hq + w.h;
        uint8_t* out = static_cast<uint8_t*>(a.o) + 2 * row_offset(head, p, a.Hq, a.N, D, a.nhd);
        const uint32_t tO = tmem + 256 + D * i + ((uint32_t)(quarter * 32) << 16);
        float odd = 0.0f;  // NaN once a value is not finite
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t x[32];
          tmem_ld32p(tO + c, x);
          tmem_ld_wait();
          if (c + 32 == D) {  // O_i is read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.o_free[i]);
          }
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float f = __uint_as_float(x[e]) * inv, g = __uint_as_float(x[e + 1]) * inv;
            odd = fmaf(f, 0.0f, fmaf(g, 0.0f, odd));
            y[e / 2] = pack16<T>(f, g);
          }
          if (p < w.n) {
            store_row32(out + 2 * c, y, wide);
            store_row32(out + 2 * c + 32, y + 8, wide);
          }
        }
        if (a.lse && p < w.n) a.lse[head * a.N + p] = (lm.y + log2f(lm.x)) * 0.6931471805599453f;
        uint32_t redo = __ballot_sync(0xffffffffu, odd != 0.0f && p < w.n);
        __syncwarp();
        for (; redo; redo &= redo - 1) window_row<T, D>(a, w.b, w.h, w.q0 + 128 * i + quarter * 32 + __ffs(redo) - 1);
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// A caller's 16-bit tensor as a TMA tensor (D, N, H, B), boxes of 64 channels x `rows` rows, 128-byte swizzle
bool map_window(CUtensorMap* m, const void* base, int D, int N, int H, int B, int nhd, int rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)H, (cuuint64_t)B};
  const cuuint64_t row = 2ull * D;
  const cuuint64_t strides[3] = {nhd ? H * row : row, nhd ? row : N * row, (cuuint64_t)H * N * row};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch_window_t(WindowArgs a, cudaStream_t st) {
  CUtensorMap q, k, v, kn, vn;
  if (!map_window(&q, a.q, D, a.N, a.Hq, a.B, a.nhd, 128) || !map_window(&k, a.k, D, a.N, a.Hkv, a.B, a.nhd, 128) ||
      !map_window(&v, a.v, D, a.N, a.Hkv, a.B, a.nhd, 128) ||
      !map_window(&kn, a.k, D, a.N, a.Hkv, a.B, a.nhd, kNarrow) ||
      !map_window(&vn, a.v, D, a.N, a.Hkv, a.B, a.nhd, kNarrow))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  auto kernel = attn_window_kernel<T, D>;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, WinSmem<D>::kBytes)) != cudaSuccess)
    return e;
  const int64_t items = (int64_t)a.B * a.Hq * ((a.N + 255) / 256);  // at most B Hq N < 2^31
  a.items = (int)items;
  // heads whose K and V (32 MB of the 126 MB L2) are in use at a time
  const int64_t kv = (int64_t)a.N * D * 4 / (a.Hq / a.Hkv) + 1;
  const int64_t group = (32 << 20) / kv;
  a.group = (int)(group < 1 ? 1 : group > (int64_t)a.B * a.Hq ? (int64_t)a.B * a.Hq : group);
  kernel<<<(unsigned)(items < sms ? items : sms), kWinThreads, WinSmem<D>::kBytes, st>>>(q, k, v, kn, vn, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_window(const WindowArgs& args, int is_fp16, cudaStream_t st) {
  WindowArgs a = args;
  // a window or sinks as long as the rows: plain causal attention (and smaller numbers below)
  if (a.window >= a.N || a.sinks >= a.N) a.window = 0;
  if (a.window == 0) a.sinks = 0;
  if (a.D == 128) return is_fp16 ? launch_window_t<__half, 128>(a, st) : launch_window_t<__nv_bfloat16, 128>(a, st);
  return is_fp16 ? launch_window_t<__half, 64>(a, st) : launch_window_t<__nv_bfloat16, 64>(a, st);
}

}  // namespace sage
