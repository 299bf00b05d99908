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
// every 128-key tile of K and V.  One CTA an SM takes items in turn (the next
// item's loads and first products run under the last one's softmax and output);
// which, it learns from the hardware's launch queue (clc_try_cancel: the grid has
// a CTA an item, and a running one takes the place of one that has not started).
// 512 threads in four warpgroups:
//   WG0, 1  softmax of row tile 0 and 1 (thread = row = TMEM lane)
//   WG2     output of both tiles
//   WG3     warp 0: TMA producer; warps 1, 2: MMA issuers of row tile 0 and 1 (one
//           thread each); warp 3: takes the items
// A step of a row tile is 64 keys: S = Q K^T, softmax, O += P V.  TMEM (512
// columns): two buffers of S a row tile, at 128 i + 64 b, with P (16 bit, the A
// operand of P V) over the first half of its S; O_i at 256 + D i.  S of the next
// step is computed while the softmax works on this one.  (Steps of 128 keys, whose
// S fills the columns that both buffers have here, left the softmax waiting 1400 of
// 4000 cycles for P V and the next S; now it waits 300 of 1880.  N = 64 costs the
// Q K^T a third of its rate: A and B then take 6 KB of shared memory for 32 cycles
// of products.)
// Each row tile has an issuing warp of its own: one thread that polled for both
// spent longer on its bookkeeping (some 2500 cycles for 128 keys) than the tensor
// core on the products.  The exponentials are the MUFU's alone: a polynomial on
// the FMA pipe for an eighth to three quarters of them made no call faster.
//
// Bound: the two chains of S, softmax and P V.  A step takes 1880 cycles, 1260 of
// them products of both row tiles (N = 64 counted at its real rate), 1020
// exponentials.  B4 H32 N4096 d128, window 1024, 4 sinks: 0.28 ms, 860 TFLOP/s of
// visible pairs; 32 heads on 8, N8192, window 4096: 0.36 ms, 1150 TFLOP/s, 69% of
// a large cuBLAS product: a few hundred calls from idle.  Called for seconds, 0.33
// and 0.42 ms: the power limit then holds the SM clock at 1575 and 1650 MHz of 1965.
//
// Keys a row does not see are -inf before the maximum, so their weights are
// exact zeros; a NaN or infinity in such a key's V still makes 0 x inf = NaN in
// the product.  A row whose output is not finite is noted, and once the CTA's
// last item is done (its waits are over, so this may take any time) it is
// computed again over its visible keys alone (window_row) if one of its steps
// held such a key.  A CTA with a row to do again takes no more items, so that
// its notes stay few; the hardware starts the others on CTAs of their own.  Rows
// of V behind a sequence's end (padding, which may hold anything) are zeroed in
// shared memory first.
#include <climits>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "serving.cuh"

namespace sage {

namespace {

constexpr int kWinThreads = 512;
constexpr int kStep = 64;              // keys of a step; rows of a half key tile (few sinks)
constexpr float kWinSlack = 8.0f;      // log2 of the largest weight over that of m, before O is rescaled
// log2 of m's own weight.  P has 16 bits; fp16 ends at 2^-24 and at 2^16, so the weights go up to 2^(8 + 7), and what a
// key loses there is at most 2^-32 of the heaviest (without the 7, 2^-25: keys 2^-24.5 as heavy came out 41% heavier).
template <typename T>
constexpr float kWinLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;
// Items of which an output warp may have rows to do again: the first, and the three that may be on their way by then
// (the ring of items holds two, and the one behind them is asked for before they are read)
constexpr int kAgain = 4;
template <int D>
struct WinSmem {
  static constexpr uint32_t kTileBytes = 128 * D * 2;
  static constexpr int kRing = D == 128 ? 5 : 8;  // K and V tiles in turn
  static constexpr uint32_t oRing = 2 * kTileBytes;
  static constexpr uint32_t oL = oRing + kRing * kTileBytes;  // float2[2][128]: l, sm_scale log2(e) m - kWinLift
  static constexpr uint32_t oItem = oL + 2 * 128 * 8;         // WinItem[2], then the launch queue's answer
  static constexpr uint32_t oAgain = oItem + 2 * 32 + 16;     // WinAgain[4][kAgain], then their numbers
  static constexpr uint32_t oBar = oAgain + 4 * kAgain * 16 + 16;
  static constexpr uint32_t kBars = 2 * kRing + 1 + 2 * 13;
  static constexpr uint32_t oTmem = oBar + 8 * kBars;
  static constexpr uint32_t kBytes = oTmem + 16;
  static_assert(kBytes <= 227 * 1024, "window attention buffers exceed the shared memory of one CTA");
};

// The key tiles of a work item: sink tiles [0, ns) with keys 128 j.., then the
// tiles of the window, keys 128 (t0 + j - ns)...
struct __align__(16) WinItem {
  int b, h, q0, n;
  int ns, t0, nt;  // nt: key tiles of the item; 0: its rows are behind the sequence; -1: no more items
  int narrow;      // the sink tile that is loaded by half, or -1
};
// The steps of row tile i: halves u of key tiles (u / 2), from `first` on, `lo` after `sink`, up to `end`.
// Steps whose keys no row sees are left out.
struct WinSteps {
  int first, sink, lo, end;
  __device__ __forceinline__ WinSteps(const WindowArgs& a, const WinItem& w, int i) {
    const int q0 = w.q0 + 128 * i, lead = q0 - a.window + 1;  // lead: first key of the window
    const int tile = w.t0 > 0 && lead > 0 ? lead / 128 : 0;
    lo = 2 * (w.ns + tile - w.t0) + (w.t0 > 0 && lead - 128 * tile >= kStep ? 1 : 0);
    sink = w.ns > 0 ? (a.sinks + kStep - 1) / kStep : -1;
    end = q0 < w.n ? 2 * (w.ns + q0 / 128 - w.t0) + (w.n - q0 <= kStep ? 1 : 2) : 0;
    first = q0 < w.n ? (w.ns > 0 ? 0 : lo) : 0;
  }
  __device__ __forceinline__ int next(int u) const { return u + 1 == sink ? lo : u + 1; }
};
__device__ __forceinline__ int win_key(const WinItem& w, int u) {  // first key of a step
  return kStep * u + (u >= 2 * w.ns ? 128 * (w.t0 - w.ns) : 0);
}
// Which steps of the row tile at p0 hold keys that one of its rows does not see: from `diagonal` on, keys behind its
// first row; before `whole`, keys that its last row's window leaves out, unless the step is one of the first
// `whole_sinks`
struct WinMask {
  int diagonal, whole_sinks, whole;
  __device__ __forceinline__ WinMask(const WindowArgs& a, const WinItem& w, int p0) {
    const int out = p0 + 128 - a.window - 128 * (w.t0 - w.ns);
    diagonal = 2 * (w.ns + p0 / 128 - w.t0);
    whole_sinks = a.sinks / kStep;
    whole = a.window > 0 && p0 + 128 > a.window ? (out + kStep - 1) / kStep : 0;
  }
  __device__ __forceinline__ bool operator()(int u) const { return u >= diagonal || (u >= whole_sinks && u < whole); }
};
// the low n bits (n taken as the nearest of 0 and 32)
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// which of the keys key0 + 32 x + 0..31 row p sees: columns c <= hi and (c >= lo or c < sk) of the step
__device__ __forceinline__ uint32_t win_sees(const WindowArgs& a, int p, int key0, int x) {
  const int hi = p - key0, lo = a.window > 0 ? hi - a.window + 1 : INT_MIN, sk = a.sinks - key0;
  return low_bits(hi + 1 - 32 * x) & (~low_bits(lo - 32 * x) | low_bits(sk - 32 * x));
}
// Rows to do again, of a warp's quarter of an item's row tiles
struct __align__(16) WinAgain {
  int bh, q0;
  uint32_t rows[2];
};
static_assert(sizeof(WinItem) == 32, "items are passed through shared memory as two 16-byte words");

// rows q0.. of head bh = b Hq + h
__device__ __forceinline__ WinItem win_rows(const WindowArgs& a, uint32_t bh, int q0) {
  WinItem w;
  w.b = bh / a.Hq;
  w.h = bh - w.b * a.Hq;
  w.q0 = q0;
  w.n = a.lens ? min(max(__ldg(a.lens + w.b), 0), a.N) : a.N;
  const int lead = w.q0 - a.window + 1;
  w.t0 = a.window > 0 && lead > 0 ? lead / 128 : 0;
  if (a.sinks > 128 * w.t0) w.t0 = 0;  // the sinks reach into the window's tiles: every tile from 0 on
  w.ns = w.t0 > 0 ? (a.sinks + 127) / 128 : 0;
  w.nt = w.q0 >= w.n ? 0 : w.ns + w.q0 / 128 - w.t0 + (w.q0 + 128 < w.n ? 2 : 1);
  w.narrow = w.ns > 0 && a.sinks - 128 * (w.ns - 1) <= kStep ? w.ns - 1 : -1;
  return w;
}
__device__ __forceinline__ WinItem win_item(const WindowArgs& a, uint32_t idx) {
  // heads in groups whose K and V stay in L2 while every pair of their rows runs, heaviest rows first
  const uint32_t per = a.group * a.pairs, g = idx / per, in = idx - g * per;
  const uint32_t heads = min((uint32_t)a.group, (uint32_t)(a.B * a.Hq) - g * a.group);
  const uint32_t pair = in / heads, bh = g * a.group + in - pair * heads;
  return win_rows(a, bh, 256 * (a.pairs - 1 - (int)pair));
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

// Of 32 rows of row tile i of an item, computes those of `rows` again whose steps held a NaN or an infinity in the V of
// a key that the row does not see; lane = row.  (What a row does see reached its output as it should.)
template <typename T, int D>
__device__ __forceinline__ void window_again(const WindowArgs& a, const WinItem& w, int i, int quarter, uint32_t rows) {
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  constexpr int LR = D / 8, RP = 32 / LR;  // lanes of a row of V, rows of a load
  const int lane = threadIdx.x & 31, hk = w.h / (a.Hq / a.Hkv);
  const int p0 = w.q0 + 128 * i, first = p0 + 32 * quarter;
  const WinSteps st(a, w, i);
  const WinMask masked(a, w, p0);
  bool again = false;
  for (int u = st.first; u != st.end; u = st.next(u)) {
    if (!masked(u)) continue;
    const int key0 = win_key(w, u);
#pragma unroll 1
    for (int x = 0; x < kStep / 32; ++x) {
      uint32_t bad = 0;  // of 32 keys
#pragma unroll 8
      for (int r = 0; r < 32; r += RP) {
        const int j = key0 + 32 * x + r + lane / LR;
        uint4 z = make_uint4(0, 0, 0, 0);  // (behind the end: zeroed before the product)
        if (j < w.n)
          z = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) +
                                             row_offset((int64_t)w.b * a.Hkv + hk, j, a.Hkv, a.N, D, a.nhd))[lane % LR];
        const uint32_t y[4] = {z.x, z.y, z.z, z.w};
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= (y[e] & kExp) == kExp || (y[e] >> 16 & kExp) == kExp;
        const uint32_t all = __ballot_sync(0xffffffffu, odd);
#pragma unroll
        for (int g = 0; g < RP; ++g)
          if (all >> (g * LR) & ((1u << LR) - 1u)) bad |= 1u << (r + g);
      }
      again |= (bad & ~win_sees(a, first + lane, key0, x)) != 0;
    }
  }
  for (rows &= __ballot_sync(0xffffffffu, again); rows; rows &= rows - 1)
    window_row<T, D>(a, w.b, w.h, first + __ffs(rows) - 1);
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
  uint64_t* kv_empty;  // [ring]  the products of a row tile that read the slot retired (one arrival a row tile)
  uint64_t* part;      // a tile of V that ends behind the sequence landed (its producer zeroes those rows)
  uint64_t* q_full;    // [2]
  uint64_t* q_empty;   // [2]  the item's last Q K^T of tile i retired
  uint64_t* s_full;    // [tile][buffer]  Q K^T retired
  uint64_t* p_full;    // [tile][buffer]  P written (one arrival a warp)
  uint64_t* pv_done;   // [2]  a P V of tile i retired
  uint64_t* o_full;    // [2]  the item's last P V of tile i retired
  uint64_t* o_free;    // [2]  the item's O_i, l and m have been read (one arrival a warp)
  uint64_t* l_ready;   // [2]  l and m of tile i in shared memory (one arrival a warp)
  uint64_t* mma_done;  // [2]  all tensor-core work of tile i retired
  uint64_t* item_full;   // [2]  an item is posted
  uint64_t* item_empty;  // [2]  every warp but the one that takes the items has read it
  uint64_t* item_want;   // the producer is about to finish the item
  uint64_t* answer;      // the launch queue answered
};
constexpr int kItemReaders = 15;

// A value that all lanes of the warp hold, known to be so: what it addresses can stay in uniform registers.  (An MMA
// whose descriptors come from per-thread registers takes some 100 cycles to issue, twice its run time.)
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// The next item, from the ring that the taking warp fills: false without one or if the wait gave up
__device__ __forceinline__ bool win_next(const WinItem* ring, const WinBars& bar, uint32_t nth, WinItem& w) {
  const uint32_t s = nth & 1;
  if (!mbar_wait_warp(&bar.item_full[s], (nth >> 1) & 1)) return false;
  const uint4* p = reinterpret_cast<const uint4*>(ring + s);
  const uint4 x = p[0], y = p[1];
  w.b = uniform(x.x), w.h = uniform(x.y), w.q0 = uniform(x.z), w.n = uniform(x.w);
  w.ns = uniform(y.x), w.t0 = uniform(y.y), w.nt = uniform(y.z), w.narrow = uniform(y.w);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.item_empty[s]);
  return w.nt >= 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWinThreads, 1)
    attn_window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKn,
                       const __grid_constant__ CUtensorMap tmVn, const __grid_constant__ WindowArgs a) {
  using L = WinSmem<D>;
  constexpr int R = L::kRing;
  constexpr uint32_t kF16 = std::is_same<T, __half>::value ? 0u : 1u;  // operand format: fp16 or bf16
  constexpr uint32_t kTransB = 1u << 16;                               // B with its N dimension contiguous
  constexpr uint32_t kIdescQK = make_idesc(1, kF16, kF16, 128, kStep);
  constexpr uint32_t kIdescPV = make_idesc(1, kF16, kF16, 128, D) | kTransB;
  constexpr uint32_t kTmemCols = 512;

  extern __shared__ __align__(1024) uint8_t smem_win[];
  uint8_t* sQ = smem_win;
  uint8_t* ring = smem_win + L::oRing;
  float2* s_l = reinterpret_cast<float2*>(smem_win + L::oL);
  WinItem* items = reinterpret_cast<WinItem*>(smem_win + L::oItem);
  WinAgain* again = reinterpret_cast<WinAgain*>(smem_win + L::oAgain);  // [4][kAgain]: a list an output warp
  volatile uint32_t* n_again = reinterpret_cast<uint32_t*>(again + 4 * kAgain);
  WinBars bar;
  bar.kv_full = reinterpret_cast<uint64_t*>(smem_win + L::oBar);
  bar.kv_empty = bar.kv_full + R;
  bar.part = bar.kv_empty + R;
  bar.q_full = bar.part + 1;
  bar.q_empty = bar.q_full + 2;
  bar.s_full = bar.q_empty + 2;
  bar.p_full = bar.s_full + 4;
  bar.pv_done = bar.p_full + 4;
  bar.o_full = bar.pv_done + 2;
  bar.o_free = bar.o_full + 2;
  bar.l_ready = bar.o_free + 2;
  bar.mma_done = bar.l_ready + 2;
  bar.item_full = bar.mma_done + 2;
  bar.item_empty = bar.item_full + 2;
  bar.item_want = bar.item_empty + 2;
  bar.answer = bar.item_want + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem_win + L::oTmem);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, wg = warp / 4;
  if (threadIdx.x < 4) n_again[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(&bar.kv_full[s], 1);
      mbar_init(&bar.kv_empty[s], 2);
    }
    mbar_init(bar.part, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.pv_done[i], 1);
      mbar_init(&bar.o_full[i], 1);
      mbar_init(&bar.o_free[i], 4);
      mbar_init(&bar.l_ready[i], 4);
      mbar_init(&bar.mma_done[i], 1);
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_empty[i], kItemReaders);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
    }
    mbar_init(bar.item_want, 1);
    mbar_init(bar.answer, 1);
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
      WinItem w;
      for (uint32_t nth = 0; ok && win_next(items, bar, nth, w); ++nth) {
        const int hk = w.h / G;
        if (lane == 0 && w.nt == 0) mbar_arrive(bar.item_want);
        for (int j = 0; j < w.nt && ok; ++j) {
          if (lane == 0 && j == max(0, w.nt - 4)) mbar_arrive(bar.item_want);
          const bool narrow = j == w.narrow;
          const int key0 = win_key(w, 2 * j);
          const uint32_t rows = narrow ? kStep : 128, bytes = rows * D * 2, half = rows * 128;
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
                if (w.q0 + 128 * i >= w.n) continue;
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
    } else if (warp < 15) {
      // ------------------------------------------------------------ MMA issuer of row tile i
      const int i = uniform(warp) - 13;
      const uint32_t base = uniform(tmem), tS = base + 128 * i, tO = base + 256 + D * i;
      // operand descriptors: 128-byte swizzle, 8 rows every 1024 bytes; the address (16 bytes a unit) is added to
      // the low word, whose upper half for V holds the distance of the slot's halves of 64 channels
      constexpr uint32_t kHi = make_sdesc(0, 1024, kSwizzle128B) >> 32, kLo = 1u << 16;
      constexpr uint32_t kSlot = L::kTileBytes / 16, kRows = kStep * 128 / 16;  // a slot; the rows of a step
      const uint32_t q = kLo + smem_u32(sQ + i * L::kTileBytes) / 16;
      const uint32_t ring0 = smem_u32(ring) / 16;
      uint32_t s_qk = 0, s_pv = 0, n_items = 0;  // steps issued, items
      bool ok = true;
      // the ring's slots of K (and V): position, parity; the key tile there; whether it has been waited for
      struct Slots {
        uint32_t at, parity;
        int tile;
        bool ready;
        __device__ __forceinline__ void advance() {
          at += 2;
          if (at >= R) {
            at -= R;
            parity ^= 1;
          }
          ++tile;
          ready = false;
        }
      } ks = {0, 0, 0, false}, vs = {1, 0, 0, false};
      // on to key tile `to`; the tiles before it, which this row tile does not see, are released unread
      auto skip = [&](Slots& s, int to) {
        while (s.tile < to && ok) {
          ok = mbar_wait_warp(&bar.kv_full[s.at], s.parity);
          if (ok && lane == 0) mbar_arrive(&bar.kv_empty[s.at]);
          s.advance();
        }
      };
      auto ready = [&](Slots& s) {
        if (!s.ready) s.ready = ok = mbar_wait_warp(&bar.kv_full[s.at], s.parity);
        return ok;
      };
      WinItem w;
      for (uint32_t nth = 0; ok && win_next(items, bar, nth, w); ++nth) {
        const WinSteps st(a, w, i);
        const bool rows = st.end > 0;
        ks.tile = vs.tile = 0;
        // none of the item's rows are here: K and V in turn (the ring holds no third K while the first V is taken)
        for (int j = 1; !rows && j <= w.nt; ++j) {
          skip(ks, j);
          skip(vs, j);
        }
        if (!rows) continue;
        skip(ks, st.first >> 1);
        skip(vs, st.first >> 1);
        ok = ok && mbar_wait_warp(&bar.q_full[i], n_items & 1);
        int c = st.first, d = st.first;  // the next S, the next P V
        auto qk = [&] {  // S = Q K^T of step c
          const int next = st.next(c);
          const bool last = next == st.end, done = last || (next ^ c) > 1;  // of the item, of the key tile
          const uint32_t k = kLo + ring0 + ks.at * kSlot + (c & 1) * kRows;
          const uint32_t half = (ks.tile == w.narrow ? kStep : 128) * 128 / 16;  // between the slot's halves
          const uint32_t dst = tS + 64 * (s_qk & 1);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
              mma_f16(dst, q + (x / 4) * 1024 + (x % 4) * 2, k + (x / 4) * half + (x % 4) * 2, kHi, kIdescQK, x > 0);
            mma_commit(&bar.s_full[2 * i + (s_qk & 1)]);
            if (done) mma_commit(&bar.kv_empty[ks.at]);
            if (last) mma_commit(&bar.q_empty[i]);
          }
          __syncwarp();
          ++s_qk;
          c = next;
          if (done) {
            ks.advance();
            skip(ks, last ? w.nt : next >> 1);
          }
        };
        for (int x = 0; x < 2 && ok && c != st.end && ready(ks); ++x) qk();
        if (ok && n_items > 0) ok = mbar_wait_warp(&bar.o_free[i], (n_items - 1) & 1);
        while (d != st.end && ok) {
          if (!ready(vs)) break;
          const int next = st.next(d);
          const bool last = next == st.end, done = last || (next ^ d) > 1;
          const uint32_t half = (vs.tile == w.narrow ? kStep : 128) * 128 / 16;
          const uint32_t v = (half << 16) + ring0 + vs.at * kSlot + (d & 1) * kRows;
          const uint32_t p = tS + 64 * (s_pv & 1);
          if (!(ok = mbar_wait_warp(&bar.p_full[2 * i + (s_pv & 1)], (s_pv >> 1) & 1))) break;
          tc_fence_after();
          // O += P V: 16 keys are 8 columns of P and 16 rows of V
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < kStep / 16; ++x)
              mma_f16_ts(tO, p + 8 * x, v + x * 128, kHi, kIdescPV, d != st.first || x > 0);
            mma_commit(&bar.pv_done[i]);
            if (done) mma_commit(&bar.kv_empty[vs.at]);
            if (last) mma_commit(&bar.o_full[i]);
          }
          __syncwarp();
          // the S that takes P's buffer (not waited for before: the ring may not hold its K until V is free)
          if (c != st.end) {
            if (!ready(ks)) break;
            qk();
          }
          ++s_pv;
          d = next;
          if (done) {
            vs.advance();
            skip(vs, last ? w.nt : next >> 1);
          }
        }
        ++n_items;
      }
      // every tensor-core op retired before TMEM is released
      if (elect_one()) {
        mma_commit(&bar.mma_done[i]);
        mbar_wait(&bar.mma_done[i], 0);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ takes the items
      uint32_t idx = blockIdx.x, asked = 0;
      bool have = true;  // idx is an item
      auto ask = [&] {
        bool got = false;
        // (no more items with a row to do again: by the time that an output warp reads the item after one, the third
        // item after it may have been asked for, and the wait to post that one shows the note here)
        if (lane == 0 && !(n_again[0] | n_again[1] | n_again[2] | n_again[3])) {
          mbar_expect_tx(bar.answer, 16);
          clc_try_cancel(items + 2, bar.answer);
          got = mbar_wait(bar.answer, asked & 1) && clc_answer(items + 2, idx);
          fence_proxy_async_smem();  // the answer is read before the next one may land
        }
        ++asked;
        have = __shfl_sync(0xffffffffu, (int)got, 0);
        idx = __shfl_sync(0xffffffffu, idx, 0);
      };
      for (uint32_t nth = 0;; ++nth) {
        WinItem w;
        w.nt = -1;
        while (have) {
          w = win_item(a, idx);
          if (w.nt > 0 || a.zero_tail) break;
          w.nt = -1;
          ask();  // (an item without rows is passed over)
        }
        if (nth >= 2 && !mbar_wait_warp(&bar.item_empty[nth & 1], ((nth >> 1) - 1) & 1)) break;
        if (lane == 0) {
          items[nth & 1] = w;
          mbar_arrive(&bar.item_full[nth & 1]);
        }
        if (w.nt < 0) break;
        // not before the item is nearly done: an item taken early is one that an idle CTA cannot take
        if (!mbar_wait_warp(bar.item_want, nth & 1)) break;
        ask();
      }
    }
  } else if (wg < 2) {
    // ------------------------------------------------------------ softmax
    const int ti = wg, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t tO = tmem + 256 + D * ti + lanes;
    const float scale = a.scale_log2, slack = kWinSlack / scale;
    uint32_t step = 0, n_items = 0;
    bool ok = true;
    WinItem w;
    for (uint32_t nth = 0; ok && win_next(items, bar, nth, w); ++nth) {
      const WinSteps st(a, w, ti);
      if (st.end == 0) continue;
      const int p0 = w.q0 + 128 * ti, p = p0 + row;
      float m = -INFINITY, l = 0.0f;
      const WinMask masked(a, w, p0);
      for (int u = st.first; u != st.end; u = st.next(u), ++step) {
        const uint32_t tS = tmem + 128 * ti + 64 * (step & 1) + lanes;
        if (!(ok = mbar_wait_warp(&bar.s_full[2 * ti + (step & 1)], (step >> 1) & 1))) break;
        tc_fence_after();
        uint32_t s[kStep];
        tmem_ld32p(tS, s);
        tmem_ld32p(tS + 32, s + 32);
        tmem_ld_wait();
        if (masked(u)) {
          const int key0 = win_key(w, u);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t see = win_sees(a, p, key0, x);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1)) s[32 * x + e] = __float_as_uint(-INFINITY);
          }
        }
        float mx4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 4]));
#pragma unroll
        for (int e = 8; e < kStep; e += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) mx4[x] = fmax3(mx4[x], __uint_as_float(s[e + x]), __uint_as_float(s[e + 4 + x]));
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        if (m == -INFINITY) m = mx;  // nothing visible before: l = 0 and O = 0 (or unset)
        const bool grow = mx > m + slack;
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2_approx((m - mx) * scale) : 1.0f;
          if (grow) m = mx;
          l *= alpha;
          if (!(ok = mbar_wait_warp(&bar.pv_done[ti], (step - 1) & 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < D; x += 16) {
            uint32_t o[16];
            tmem_ld16p(tO + x, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16p(tO + x, o);
          }
        }
        const float ms = (m == -INFINITY ? 0.0f : m * scale) - kWinLift<T>;
        const float2 sc = make_float2(scale, scale), off = make_float2(-ms, -ms);
        float2 sum[4] = {};
#pragma unroll
        for (int x = 0; x < kStep; x += 32) {  // into P, over S
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 u = ffma2(make_float2(__uint_as_float(s[x + e]), __uint_as_float(s[x + e + 1])), sc, off);
            const float2 f = make_float2(ex2_approx(u.x), ex2_approx(u.y));
            sum[(e / 2) & 3] = fadd2(sum[(e / 2) & 3], f);
            y[e / 2] = pack16<T>(f.x, f.y);  // A of P V has V's type: one rounding, after the sum has taken f
          }
          tmem_st16p(tS + x / 2, y);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[2 * ti + (step & 1)]);
        const float2 t = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
        l += t.x + t.y;
      }
      if (!ok) break;
      // l and m for the output warps, once they have read the last item's
      if (n_items > 0 && !(ok = mbar_wait_warp(&bar.o_free[ti], (n_items - 1) & 1))) break;
      s_l[128 * ti + row] = make_float2(l, m * scale - kWinLift<T>);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.l_ready[ti]);
      ++n_items;
    }
  } else {
    // ------------------------------------------------------------ output
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const bool wide = (reinterpret_cast<uintptr_t>(a.o) & 31) == 0;
    uint32_t n_items[2] = {0, 0}, noted = 0;
    bool ok = true;
    WinItem w;
    for (uint32_t nth = 0; ok && win_next(items, bar, nth, w); ++nth) {
      uint32_t redo[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = w.q0 + 128 * i + row;
        const int64_t head = (int64_t)w.b * a.Hq + w.h;
        uint8_t* out = static_cast<uint8_t*>(a.o) + 2 * row_offset(head, p, a.Hq, a.N, D, a.nhd);
        if (a.zero_tail && p >= w.n && p < a.N) {
          if (a.zero_tail & 1)
            for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(out + 2 * c) = make_uint4(0, 0, 0, 0);
          if ((a.zero_tail & 2) && a.lse) a.lse[head * a.N + p] = 0.0f;
        }
        __syncwarp();
        if (w.q0 + 128 * i >= w.n || !ok) continue;
        if (!(ok = mbar_wait_warp(&bar.l_ready[i], n_items[i] & 1))) break;
        if (!(ok = mbar_wait_warp(&bar.o_full[i], n_items[i] & 1))) break;
        tc_fence_after();
        ++n_items[i];
        const float2 lm = s_l[128 * i + row];
        const float inv = 1.0f / lm.x;
        const uint32_t tO = tmem + 256 + D * i + ((uint32_t)(quarter * 32) << 16);
        float odd = 0.0f;  // NaN once a value is not finite
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t x[32];
          tmem_ld32p(tO + c, x);
          tmem_ld_wait();
          if (c + 32 == D) {  // O_i, l and m are read
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
        redo[i] = __ballot_sync(0xffffffffu, odd != 0.0f && p < w.n);
      }
      if (redo[0] | redo[1]) {
        if (lane == 0) {
          again[kAgain * quarter + noted] = {w.b * a.Hq + w.h, w.q0, {redo[0], redo[1]}};
          n_again[quarter] = noted + 1;
        }
        ++noted;
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
  // rows to do again: (item, row tile, quarter) in turn to the warps
  for (int x = warp; x < 8 * kAgain; x += kWinThreads / 32) {
    const int quarter = x % 4, i = x / 4 % 2, nth = x / 8;
    if (nth >= n_again[quarter]) continue;
    const WinAgain& r = again[kAgain * quarter + nth];
    const uint32_t rows = r.rows[i];
    if (rows) window_again<T, D>(a, win_rows(a, r.bh, r.q0), i, quarter, rows);
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
      !map_window(&v, a.v, D, a.N, a.Hkv, a.B, a.nhd, 128))
    return cudaErrorInvalidValue;
  kn = k, vn = v;
  if (a.sinks > 0 && (a.sinks - 1) % 128 < kStep &&
      (!map_window(&kn, a.k, D, a.N, a.Hkv, a.B, a.nhd, kStep) ||
       !map_window(&vn, a.v, D, a.N, a.Hkv, a.B, a.nhd, kStep)))
    return cudaErrorInvalidValue;
  auto kernel = attn_window_kernel<T, D>;
  static DeviceOnce once;
  const cudaError_t e = once.run([&](int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, WinSmem<D>::kBytes);
  });
  if (e != cudaSuccess) return e;
  const int64_t heads = (int64_t)a.B * a.Hq;
  a.pairs = (a.N + 255) / 256;
  a.items = (int)(heads * a.pairs);  // at most B Hq N < 2^31
  // heads whose K and V (32 MB of the 126 MB L2) are in use at a time, in groups of one size: 366 us with 8 MB, 358
  // with 32, for N 8192 on 8 kv heads; 279 us with 32 MB, 289 with 128, for B4 H32 N4096
  const int64_t kv = (int64_t)a.N * D * 4;
  int64_t groups = (heads * kv / (a.Hq / a.Hkv) + (32 << 20) - 1) >> 25;
  groups = groups < 1 ? 1 : groups > heads ? heads : groups;
  a.group = (int)((heads + groups - 1) / groups);
  kernel<<<(unsigned)a.items, kWinThreads, WinSmem<D>::kBytes, st>>>(q, k, v, kn, vn, a);
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
