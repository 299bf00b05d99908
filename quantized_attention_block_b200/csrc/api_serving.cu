// api_serving.cu -- the extern "C" entry points of the paged key-value cache,
// the single-token attention over it and the sliding-window attention:
// argument validation, workspace layout, launches.
#include <cmath>
#include <cstdint>

#include "sage.h"
#include "serving.cuh"

namespace {

using namespace sage;

// check_arch() of the current device, asked once
sage_status check_device() {
  static DeviceOnce once;
  int st = SAGE_OK;
  const cudaError_t e = once.run([&](int dev) {
    once.value[dev] = check_arch();
    return once.value[dev].load() == SAGE_ERR_CUDA ? cudaErrorUnknown : cudaSuccess;
  }, &st);
  return e != cudaSuccess ? SAGE_ERR_CUDA : (sage_status)st;
}

sage_status check_cache(const sage_kv_cache* c, const sage_kv_seqs* s) {
  if (!c || !s) return SAGE_ERR_INVALID_ARG;
  if (c->Hkv < 1 || c->Hkv > 65535 || c->n_pages < 1 || s->B < 1 || s->B > 65535 || s->max_pages < 1)
    return SAGE_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return SAGE_ERR_INVALID_ARG;
  if ((int64_t)s->max_pages * c->page_size >= (int64_t(1) << 30)) return SAGE_ERR_INVALID_ARG;
  if (c->layout != SAGE_HND && c->layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (c->quantized != 0 && c->quantized != 1) return SAGE_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return SAGE_ERR_UNSUPPORTED_HEADDIM;
  if (c->dtype != SAGE_BF16 && c->dtype != SAGE_FP16) return SAGE_ERR_UNSUPPORTED_DTYPE;
  return SAGE_OK;
}

// the pointers of the cache and the sequences
sage_status check_cache_ptrs(const sage_kv_cache* c, const sage_kv_seqs* s) {
  if (!c->k_pages || !c->v_pages || !s->table || !s->lens) return SAGE_ERR_INVALID_ARG;
  if (c->quantized && (!c->k_scale || !c->v_scale)) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
      (reinterpret_cast<uintptr_t>(c->weight) & 3u) || (reinterpret_cast<uintptr_t>(s->table) & 3u) ||
      (reinterpret_cast<uintptr_t>(s->lens) & 3u))
    return SAGE_ERR_MISALIGNED;
  return SAGE_OK;
}

CacheArgs cache_args(const sage_kv_cache* c, const sage_kv_seqs* s) {
  CacheArgs a{};
  a.k = c->k_pages;
  a.v = c->v_pages;
  a.ks = c->quantized ? c->k_scale : nullptr;
  a.vs = c->quantized ? c->v_scale : nullptr;
  a.weight = c->weight;
  a.H = c->Hkv;
  a.D = c->d;
  while ((1 << a.page_log2) < c->page_size) ++a.page_log2;
  a.n_pages = c->n_pages;
  a.page_stride = (int64_t)c->Hkv * c->page_size * c->d;
  a.hs = c->layout == SAGE_HND ? (int64_t)c->page_size * c->d : c->d;
  a.rs = c->layout == SAGE_HND ? c->d : (int64_t)c->Hkv * c->d;
  a.table = s->table;
  a.lens = s->lens;
  a.B = s->B;
  a.max_pages = s->max_pages;
  a.cap = s->max_pages * c->page_size;
  return a;
}

sage_status check_decode(const sage_kv_cache* c, const sage_kv_seqs* s, const sage_decode_params* p) {
  const sage_status st = check_cache(c, s);
  if (st != SAGE_OK) return st;
  if (!p || p->Hq < 1 || p->Hq % c->Hkv != 0 || p->window < 0 || p->sinks < 0) return SAGE_ERR_INVALID_ARG;
  if ((int64_t)s->B * p->Hq >= (int64_t(1) << 31)) return SAGE_ERR_INVALID_ARG;
  if (std::isnan(p->sm_scale) || std::isinf(p->sm_scale)) return SAGE_ERR_INVALID_ARG;
  return SAGE_OK;
}

int group_tiles(int G) { return G <= 8 ? 1 : (G + kMaxGroup - 1) / kMaxGroup; }

struct DecodeLayout {
  size_t prefix, part_m, part_l, part_o, lse2, scores, total;
  int64_t score_cap;
  bool direct;
};

DecodeLayout decode_layout(const sage_kv_cache* c, const sage_kv_seqs* s, const sage_decode_params* p) {
  DecodeLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const int64_t blocks = most_blocks((int64_t)s->max_pages * c->page_size, p->window, p->sinks);
  L.direct = decode_direct((int64_t)s->B * c->Hkv * group_tiles(p->Hq / c->Hkv), blocks);
  L.prefix = take(L.direct ? 1 : 8 * ((size_t)s->B + 1));
  if (!L.direct) {
    L.part_m = take(4 * (size_t)(2 * kDecodeCtas * kMaxGroup));
    L.part_l = take(4 * (size_t)(2 * kDecodeCtas * kMaxGroup));
    L.part_o = take(4 * (size_t)(2 * kDecodeCtas * kMaxGroup) * c->d);
  }
  if (c->weight) {
    L.score_cap = blocks * kBlk;
    L.lse2 = take(4 * (size_t)s->B * p->Hq);
    L.scores = take(4 * (size_t)s->B * p->Hq * (size_t)L.score_cap);
  }
  L.total = off;
  return L;
}

float scale_or_default(float sm_scale, int d) { return sm_scale > 0.0f ? sm_scale : 1.0f / std::sqrt((float)d); }

}  // namespace

extern "C" {

sage_status sage_kv_append(const void* k, const void* v, const int32_t* n_new, const float* km, int32_t T,
                           int32_t layout, const sage_kv_cache* c, const sage_kv_seqs* s, void* stream) {
  sage_status st = check_cache(c, s);
  if (st != SAGE_OK) return st;
  if (T < 0 || (layout != SAGE_HND && layout != SAGE_NHD) || (km && !c->quantized)) return SAGE_ERR_INVALID_ARG;
  if ((int64_t)s->B * c->Hkv * T >= (int64_t(1) << 31)) return SAGE_ERR_INVALID_ARG;
  if ((T > 0 && (!k || !v))) return SAGE_ERR_INVALID_ARG;
  if ((st = check_cache_ptrs(c, s)) != SAGE_OK) return st;
  if (!aligned16(k) || !aligned16(v) || !aligned16(km) || (reinterpret_cast<uintptr_t>(n_new) & 3u))
    return SAGE_ERR_MISALIGNED;
  if ((st = check_device()) != SAGE_OK) return st;
  AppendArgs a{};
  a.c = cache_args(c, s);
  a.k = k;
  a.v = v;
  a.n_new = n_new;
  a.km = km;
  a.T = T;
  a.nhd = layout == SAGE_NHD;
  a.quantized = c->quantized;
  a.is_fp16 = c->dtype == SAGE_FP16;
  return from_cuda(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

size_t sage_decode_workspace_bytes(const sage_kv_cache* c, const sage_kv_seqs* s, const sage_decode_params* p) {
  if (check_decode(c, s, p) != SAGE_OK) return 0;
  return decode_layout(c, s, p).total;
}

sage_status sage_attn_decode(const void* q, void* o, float* lse, const float* km, const sage_kv_cache* c,
                             const sage_kv_seqs* s, const sage_decode_params* p, void* workspace,
                             size_t workspace_bytes, void* stream) {
  sage_status st = check_decode(c, s, p);
  if (st != SAGE_OK) return st;
  if (!q || !o || !workspace || (km && !c->quantized)) return SAGE_ERR_INVALID_ARG;
  if ((st = check_cache_ptrs(c, s)) != SAGE_OK) return st;
  if (!aligned16(q) || !aligned16(o) || !aligned16(km) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SAGE_ERR_MISALIGNED;
  const DecodeLayout L = decode_layout(c, s, p);
  if (workspace_bytes < L.total) return SAGE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device()) != SAGE_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeArgs a{};
  a.c = cache_args(c, s);
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.km = km;
  a.Hq = p->Hq;
  a.G = p->Hq / c->Hkv;
  a.GT = group_tiles(a.G);
  a.direct = L.direct;
  a.window = p->window;
  a.sinks = p->sinks;
  a.q_fp16 = c->dtype == SAGE_FP16;
  a.sm_scale = scale_or_default(p->sm_scale, c->d);
  a.scale_log2 = (float)((double)a.sm_scale * 1.4426950408889634);
  a.prefix = reinterpret_cast<long long*>(ws + L.prefix);
  a.part_m = reinterpret_cast<float*>(ws + L.part_m);
  a.part_l = reinterpret_cast<float*>(ws + L.part_l);
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  if (c->weight) {
    a.lse2 = reinterpret_cast<float*>(ws + L.lse2);
    a.scores = reinterpret_cast<float*>(ws + L.scores);
    a.score_cap = L.score_cap;
  }
  return from_cuda(launch_attn_decode(a, c->quantized, static_cast<cudaStream_t>(stream)));
}

sage_status sage_kv_evict(const sage_kv_cache* c, const sage_kv_seqs* s, const int32_t* dst_table, int32_t dst_pages,
                          int32_t keep, int32_t sinks, int32_t recent, int32_t* new_lens, int32_t* kept,
                          void* stream) {
  sage_status st = check_cache(c, s);
  if (st != SAGE_OK) return st;
  if (!dst_table || !new_lens || !kept || !c->weight) return SAGE_ERR_INVALID_ARG;
  if (keep < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep) return SAGE_ERR_INVALID_ARG;
  if (dst_pages < 1 || (int64_t)dst_pages * c->page_size < keep) return SAGE_ERR_INVALID_ARG;
  if (dst_table == s->table || new_lens == s->lens) return SAGE_ERR_INVALID_ARG;
  if ((int64_t)s->B * c->Hkv >= (int64_t(1) << 31)) return SAGE_ERR_INVALID_ARG;
  if ((st = check_cache_ptrs(c, s)) != SAGE_OK) return st;
  if ((reinterpret_cast<uintptr_t>(dst_table) & 3u) || (reinterpret_cast<uintptr_t>(new_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(kept) & 3u))
    return SAGE_ERR_MISALIGNED;
  if ((st = check_device()) != SAGE_OK) return st;
  EvictArgs a{};
  a.c = cache_args(c, s);
  a.dst_table = dst_table;
  a.dst_pages = dst_pages;
  a.keep = keep;
  a.sinks = sinks;
  a.recent = recent;
  a.new_lens = new_lens;
  a.kept = kept;
  a.quantized = c->quantized;
  return from_cuda(launch_kv_evict(a, static_cast<cudaStream_t>(stream)));
}

sage_status sage_attn_window_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                                 const int32_t* lens, const sage_window_params* p, void* stream) {
  if (!p) return SAGE_ERR_INVALID_ARG;
  if (p->B < 1 || p->Hq < 1 || p->Hkv < 1 || p->N < 1 || p->Hq % p->Hkv != 0) return SAGE_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SAGE_ERR_UNSUPPORTED_HEADDIM;
  if (p->dtype != SAGE_BF16 && p->dtype != SAGE_FP16) return SAGE_ERR_UNSUPPORTED_DTYPE;
  if (p->layout != SAGE_HND && p->layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (p->window < 0 || p->sinks < 0 || (p->zero_tail & ~3)) return SAGE_ERR_INVALID_ARG;
  if (std::isnan(p->sm_scale) || std::isinf(p->sm_scale)) return SAGE_ERR_INVALID_ARG;
  if ((int64_t)p->B * p->Hq * p->N >= (int64_t(1) << 31)) return SAGE_ERR_INVALID_ARG;
  if (!q || !k || !v || !o) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(lens) & 3u))
    return SAGE_ERR_MISALIGNED;
  sage_status st = check_device();
  if (st != SAGE_OK) return st;
  WindowArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  a.lens = lens;
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.N = p->N;
  a.D = p->d;
  a.nhd = p->layout == SAGE_NHD;
  a.window = p->window;
  a.sinks = p->sinks;
  a.zero_tail = lens ? p->zero_tail : 0;
  a.sm_scale = scale_or_default(p->sm_scale, p->d);
  a.scale_log2 = (float)((double)a.sm_scale * 1.4426950408889634);
  return from_cuda(launch_attn_window(a, p->dtype == SAGE_FP16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
