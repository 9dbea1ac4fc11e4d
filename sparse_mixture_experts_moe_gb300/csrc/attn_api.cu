// C ABI of the attention and cache operators (include/moe.h): host-side validation, workspace layout and
// the choice of kernel. As in api.cu, every argument is checked before any CUDA call.
#include <cmath>
#include <cstring>

#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int elem_bytes(int dt) { return dt == MOE_DTYPE_BF16 ? 2 : 4; }
inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool dtype_ok(int dt) { return dt == MOE_DTYPE_F32 || dt == MOE_DTYPE_BF16; }
bool heads_ok(int H, int Hkv, int D) {
  return H >= 1 && Hkv >= 1 && H <= 65535 && H % Hkv == 0 && D >= 8 && D <= 256 && D % 8 == 0;
}
bool scale_ok(float s) { return s > 0.f && std::isfinite(s * 1.4426950408889634f); }  // (as the kernels take it)
// Rows of `inner` dense elements every `stride` elements, each row 16-byte aligned; strides below 2^40.
bool stride_ok(int64_t stride, long long inner, int dt) {
  return stride >= inner && stride < (1ll << 40) && stride * elem_bytes(dt) % 16 == 0;
}
bool workspace_ok(const void* ws, size_t have, size_t need) {
  return ws != nullptr && aligned16(ws) && have >= need;
}
// The scratch memory of an attention call: apart, or the workspace from its header on.
struct Scratch {
  float* at;
  size_t bytes;
};
bool scratch_of(void* ws, size_t ws_bytes, void* scratch, size_t scratch_bytes, Scratch* s) {
  if (!workspace_ok(ws, ws_bytes, kWsHeaderBytes) || !aligned16(scratch) || (scratch == nullptr && scratch_bytes != 0)) return false;
  s->at = static_cast<float*>(scratch != nullptr ? scratch : static_cast<uint8_t*>(ws) + kWsHeaderBytes);
  s->bytes = scratch != nullptr ? scratch_bytes : ws_bytes - kWsHeaderBytes;
  return true;
}

// Keys of a sequence, so that a block's end is still a 32-bit position.
constexpr long long kMostKeys = (1ll << 31) - 256;
bool cache_sizes_ok(const moe_kv_cache* c) {
  if (c == nullptr || !dtype_ok(c->dt) || !heads_ok(c->H_kv, c->H_kv, c->D)) return false;
  if (c->n_layers < 1 || c->n_layers > 4096 || c->n_pages < 1 || c->n_pages >= (1 << 30)) return false;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0) return false;
  if (c->n_slots < 1 || c->n_slots >= (1 << 30) || c->table_width < 1 || (long long)c->n_slots * c->table_width >= (1ll << 31)) return false;
  if ((long long)c->table_width * c->page_size > kMostKeys) return false;
  // the rows of a layer are numbered with 32 bits
  return (long long)c->n_pages * c->H_kv * c->page_size < (1ll << 31);
}
bool cache_ok(const moe_kv_cache* c) {
  return cache_sizes_ok(c) && c->k != nullptr && c->v != nullptr && c->table != nullptr && c->lens != nullptr &&
         c->refs != nullptr && aligned16(c->k) && aligned16(c->v);
}
CacheView view_of(const moe_kv_cache* c) {
  CacheView v;
  v.k = c->k; v.v = c->v; v.table = c->table; v.lens = c->lens; v.refs = c->refs;
  v.n_layers = c->n_layers; v.n_pages = c->n_pages; v.page_size = c->page_size;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c->page_size) ++v.page_shift;
  v.n_slots = c->n_slots; v.width = c->table_width; v.Hkv = c->H_kv; v.D = c->D; v.dt = c->dt;
  return v;
}

struct CacheLayout {
  size_t claim_d, claim_s, counts, zeroed, entry, entry2, freel, copies, map, end;
  explicit CacheLayout(const moe_kv_cache* c) {
    const size_t slots = c->n_slots, pages = c->n_pages;
    size_t o = align256(kWsHeaderBytes);
    claim_d = o; o += align256(slots * 4);
    claim_s = o; o += align256(slots * 4);
    counts = o; o += 256;
    zeroed = o;  // everything up to here starts at zero
    entry = o; o += align256(slots * 16);
    entry2 = o; o += align256(slots * 16);
    freel = o; o += align256(pages * 4);
    copies = o; o += align256((slots > pages ? slots : pages) * 8);
    map = o; o += align256(pages * 4);
    end = o;
  }
};
CacheWs cache_ws(const moe_kv_cache* c, void* ws) {
  const CacheLayout L(c);
  uint8_t* b = static_cast<uint8_t*>(ws);
  CacheWs w;
  w.status = reinterpret_cast<int*>(b);
  w.claim_d = reinterpret_cast<int32_t*>(b + L.claim_d);
  w.claim_s = reinterpret_cast<int32_t*>(b + L.claim_s);
  w.counts = reinterpret_cast<int32_t*>(b + L.counts);
  w.entry = reinterpret_cast<int4*>(b + L.entry);
  w.entry2 = reinterpret_cast<int4*>(b + L.entry2);
  w.freel = reinterpret_cast<int32_t*>(b + L.freel);
  w.copies = reinterpret_cast<int2*>(b + L.copies);
  w.map = reinterpret_cast<int32_t*>(b + L.map);
  return w;
}
bool cache_call_ok(const moe_kv_cache* c, const void* ws, size_t ws_bytes) {
  return cache_ok(c) && workspace_ok(ws, ws_bytes, CacheLayout(c).end);
}

// What moe_cache_plan writes: the descriptors, and the cache that they describe.
struct CachePlan {
  CacheMaps maps;
  const void *k, *v;
  int n_layers, n_pages, page_size, H_kv, D, dt;
};
bool plan_holds(const CachePlan& p, const moe_kv_cache* c) {
  return p.k == c->k && p.v == c->v && p.n_layers == c->n_layers && p.n_pages == c->n_pages &&
         p.page_size == c->page_size && p.H_kv == c->H_kv && p.D == c->D && p.dt == c->dt;
}
bool planned(const moe_kv_cache* c) { return c->dt == MOE_DTYPE_BF16 && c->D <= 128; }

size_t decode_ws_bytes(int n, int H, int D) {
  return kWsHeaderBytes + align256((size_t)decode_pieces((long long)n * H) * (D + 2) * 4);
}

size_t prompt_ws_bytes(long long rows, int splits, int D) {
  return kWsHeaderBytes + (splits > 1 ? align256((size_t)rows * splits * (D + 2) * 4) : 0);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_attention_prompt_workspace_bytes(int n_seqs, int Tq, int Tkv, int H, int H_kv, int D, moe_dtype dt) {
  if (!dtype_ok(dt) || !heads_ok(H, H_kv, D) || n_seqs < 0 || Tq < 0 || Tkv < 0 ||
      (long long)Tq * H + (long long)n_seqs * H_kv >= (1ll << 31))
    return 0;
  const bool tc = dt == MOE_DTYPE_BF16 && D <= 128 && Tq > 0;
  return prompt_ws_bytes((long long)Tq * H, tc ? attn_prompt_splits(n_seqs, Tq, Tkv, H, H_kv) : 1, D);
}

moe_status moe_attention_prompt(const void* q, const void* k, const void* v, const int32_t* q_offsets,
                                const int32_t* kv_offsets, int n_seqs, int Tq, int Tkv, int H, int H_kv, int D,
                                int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t out_stride, float scale,
                                int flags, moe_dtype dt, void* out, float* lse, void* workspace, size_t ws_bytes,
                                void* stream) {
  return moe_attention_prompt_ex(q, k, v, q_offsets, kv_offsets, n_seqs, Tq, Tkv, H, H_kv, D, q_stride, k_stride, v_stride,
                                 out_stride, scale, flags, dt, out, lse, workspace, ws_bytes, nullptr, 0, stream);
}

moe_status moe_attention_prompt_ex(const void* q, const void* k, const void* v, const int32_t* q_offsets,
                                   const int32_t* kv_offsets, int n_seqs, int Tq, int Tkv, int H, int H_kv, int D,
                                   int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t out_stride,
                                   float scale, int flags, moe_dtype dt, void* out, float* lse, void* workspace,
                                   size_t ws_bytes, void* scratch, size_t scratch_bytes, void* stream) {
  if (!dtype_ok(dt) || !heads_ok(H, H_kv, D) || !scale_ok(scale) || (flags & ~MOE_ATTN_CAUSAL) != 0)
    return MOE_ERR_INVALID_ARG;
  if (n_seqs < 0 || Tq < 0 || Tkv < 0 || (Tq > 0 && n_seqs == 0)) return MOE_ERR_INVALID_ARG;
  if ((kv_offsets == nullptr && Tkv != Tq) || Tkv > kMostKeys) return MOE_ERR_INVALID_ARG;
  // rows and work items are numbered with 32 bits
  if ((long long)Tq * H + (long long)n_seqs * H_kv >= (1ll << 31)) return MOE_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, (long long)H * D, dt) || !stride_ok(out_stride, (long long)H * D, dt) ||
      !stride_ok(k_stride, (long long)H_kv * D, dt) || !stride_ok(v_stride, (long long)H_kv * D, dt))
    return MOE_ERR_INVALID_ARG;
  Scratch room;
  if (!scratch_of(workspace, ws_bytes, scratch, scratch_bytes, &room)) return MOE_ERR_INVALID_ARG;
  if (Tq == 0) return MOE_OK;
  if (q == nullptr || out == nullptr || q_offsets == nullptr || (Tkv > 0 && (k == nullptr || v == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  PromptArgs a;
  a.q = q; a.k = k; a.v = v;
  a.qo = q_offsets;
  a.ko = kv_offsets != nullptr ? kv_offsets : q_offsets;
  a.n = n_seqs; a.Tq = Tq; a.Tkv = Tkv; a.H = H; a.Hkv = H_kv; a.D = D;
  a.qs = q_stride; a.ks = k_stride; a.vs = v_stride; a.os = out_stride;
  a.scale = scale;
  a.causal = (flags & MOE_ATTN_CAUSAL) != 0;
  a.dt = dt;
  a.out = out; a.lse = lse;
  a.status = static_cast<int*>(workspace);
  a.timeout_ns = wait_timeout_ns() + replace_time(Tkv);
  // bf16 heads of up to 128 elements go to tcgen05 (a tile of longer ones does not fit in TMEM); its copies need a key.
  if (dt == MOE_DTYPE_BF16 && D <= 128 && Tkv > 0) {
    bind_primary_context();
    int splits = attn_prompt_splits(n_seqs, Tq, Tkv, H, H_kv);
    if (room.bytes < prompt_ws_bytes((long long)Tq * H, splits, D) - kWsHeaderBytes) splits = 1;
    return cuda_status(launch_attn_prompt_tc(a, splits, room.at, (cudaStream_t)stream));
  }
  return cuda_status(dt == MOE_DTYPE_BF16 ? launch_attn_prompt_mma(a, (cudaStream_t)stream)
                                          : launch_attn_prompt_simt(a, (cudaStream_t)stream));
}

size_t moe_attention_workspace_bytes(int n, int H, int D) {
  if (n < 0 || !heads_ok(H, H, D) || (long long)n * H >= (1ll << 31)) return 0;
  return decode_ws_bytes(n, H, D);
}

moe_status moe_attention_decode(const moe_kv_cache* cache, int layer, const void* q, const int32_t* slots, int n, int H,
                                int64_t q_stride, int64_t out_stride, int shared_len, float scale, void* out,
                                float* lse, void* workspace, size_t ws_bytes, void* stream) {
  return moe_attention_decode_ex(cache, layer, q, slots, n, H, q_stride, out_stride, shared_len, scale, out, lse, workspace,
                                 ws_bytes, nullptr, 0, stream);
}

moe_status moe_attention_decode_ex(const moe_kv_cache* cache, int layer, const void* q, const int32_t* slots, int n, int H,
                                   int64_t q_stride, int64_t out_stride, int shared_len, float scale, void* out,
                                   float* lse, void* workspace, size_t ws_bytes, void* scratch, size_t scratch_bytes,
                                   void* stream) {
  if (!cache_ok(cache) || layer < 0 || layer >= cache->n_layers || n < 0) return MOE_ERR_INVALID_ARG;
  if (!heads_ok(H, cache->H_kv, cache->D) || !scale_ok(scale) || (long long)n * H >= (1ll << 31))
    return MOE_ERR_INVALID_ARG;
  if (shared_len < 0 || shared_len % cache->page_size != 0 ||
      shared_len > (long long)cache->table_width * cache->page_size)
    return MOE_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, (long long)H * cache->D, cache->dt) ||
      !stride_ok(out_stride, (long long)H * cache->D, cache->dt))
    return MOE_ERR_INVALID_ARG;
  Scratch room;
  if (!scratch_of(workspace, ws_bytes, scratch, scratch_bytes, &room) ||
      room.bytes < decode_ws_bytes(n, H, cache->D) - kWsHeaderBytes)
    return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (q == nullptr || slots == nullptr || out == nullptr || !aligned16(q) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  DecodeArgs a;
  a.q = q; a.qs = q_stride; a.os = out_stride; a.slots = slots; a.lead = slots; a.first = 0; a.n = n; a.H = H; a.shared = shared_len;
  a.scale = scale;
  a.c = view_of(cache);
  const size_t off = (size_t)layer * a.c.layer_elems() * elem_bytes(cache->dt);
  a.k = static_cast<const uint8_t*>(cache->k) + off;
  a.v = static_cast<const uint8_t*>(cache->v) + off;
  a.out = out; a.lse = lse;
  a.part = room.at;
  a.status = static_cast<int*>(workspace);
  a.timeout_ns = wait_timeout_ns() + replace_time(shared_len);
  a.layer = layer;
  CachePlan p;
  if (cache->plan != nullptr) {
    std::memcpy(&p, cache->plan, sizeof(p));
    if (!plan_holds(p, cache)) return MOE_ERR_INVALID_ARG;
  }
  if (planned(cache)) {
    bind_primary_context();
    if (cache->plan == nullptr && !encode_cache_maps(a.c, &p.maps)) return MOE_ERR_CUDA;
    return cuda_status(launch_attn_decode_tc(a, p.maps, (cudaStream_t)stream));
  }
  return cuda_status(launch_attn_decode_simt(a, (cudaStream_t)stream));
}

size_t moe_cache_plan_bytes(void) { return sizeof(CachePlan); }

moe_status moe_cache_plan(const moe_kv_cache* cache, void* plan, size_t bytes) {
  if (!cache_ok(cache) || plan == nullptr || bytes < sizeof(CachePlan)) return MOE_ERR_INVALID_ARG;
  CachePlan p{};
  p.k = cache->k; p.v = cache->v;
  p.n_layers = cache->n_layers; p.n_pages = cache->n_pages; p.page_size = cache->page_size;
  p.H_kv = cache->H_kv; p.D = cache->D; p.dt = cache->dt;
  if (planned(cache)) {  // other caches take the CUDA cores, which need no descriptors
    bind_primary_context();
    if (!encode_cache_maps(view_of(cache), &p.maps)) return MOE_ERR_CUDA;
  }
  std::memcpy(plan, &p, sizeof(p));
  return MOE_OK;
}

size_t moe_cache_workspace_bytes(const moe_kv_cache* cache) {
  return cache_sizes_ok(cache) ? CacheLayout(cache).end : 0;
}

moe_status moe_cache_workspace_init(const moe_kv_cache* cache, void* workspace, size_t ws_bytes, void* stream) {
  if (!cache_sizes_ok(cache) || !workspace_ok(workspace, ws_bytes, CacheLayout(cache).end)) return MOE_ERR_INVALID_ARG;
  return cuda_status(cudaMemsetAsync(workspace, 0, CacheLayout(cache).zeroed, (cudaStream_t)stream));
}

moe_status moe_cache_clear(const moe_kv_cache* cache, void* stream) {
  if (!cache_ok(cache)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaMemsetAsync(cache->table, 0xff, (size_t)cache->n_slots * cache->table_width * 4, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(cache->lens, 0, (size_t)cache->n_slots * 4, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(cache->refs, 0, (size_t)cache->n_pages * 4, s);
  return cuda_status(e);
}

moe_status moe_cache_resize(const moe_kv_cache* cache, const int32_t* slots, const int32_t* new_lens, int n,
                            void* workspace, size_t ws_bytes, void* stream) {
  if (!cache_call_ok(cache, workspace, ws_bytes) || n < 0 || n > cache->n_slots) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (slots == nullptr || new_lens == nullptr) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_cache_resize(view_of(cache), cache_ws(cache, workspace), slots, new_lens, n,
                                         (cudaStream_t)stream));
}

moe_status moe_cache_fork(const moe_kv_cache* cache, const int32_t* src, const int32_t* dst, int n, void* workspace,
                          size_t ws_bytes, void* stream) {
  if (!cache_call_ok(cache, workspace, ws_bytes) || n < 0 || n > cache->n_slots) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (src == nullptr || dst == nullptr) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_cache_fork(view_of(cache), cache_ws(cache, workspace), src, dst, n, (cudaStream_t)stream));
}

moe_status moe_cache_compact(const moe_kv_cache* cache, int32_t* n_live, void* workspace, size_t ws_bytes,
                             void* stream) {
  if (!cache_call_ok(cache, workspace, ws_bytes)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_cache_compact(view_of(cache), cache_ws(cache, workspace), n_live, (cudaStream_t)stream));
}

moe_status moe_cache_copy_pages(const moe_kv_cache* cache, const int32_t* src, const int32_t* dst, int n,
                                void* workspace, size_t ws_bytes, void* stream) {
  if (!cache_call_ok(cache, workspace, ws_bytes) || n < 0 || n > cache->n_pages) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (src == nullptr || dst == nullptr) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_cache_copy(view_of(cache), cache_ws(cache, workspace), src, dst, n, (cudaStream_t)stream));
}

moe_status moe_cache_write(const moe_kv_cache* cache, int layer, const int32_t* slots, const int32_t* offsets,
                           const int32_t* pos, int n, int total, const void* k_new, const void* v_new,
                           int64_t k_stride, int64_t v_stride, void* workspace, size_t ws_bytes, void* stream) {
  if (!cache_call_ok(cache, workspace, ws_bytes) || layer < 0 || layer >= cache->n_layers) return MOE_ERR_INVALID_ARG;
  if (n < 0 || n > cache->n_slots || total < 0 || (total > 0 && n == 0)) return MOE_ERR_INVALID_ARG;
  const long long inner = (long long)cache->H_kv * cache->D;
  if (!stride_ok(k_stride, inner, cache->dt) || !stride_ok(v_stride, inner, cache->dt)) return MOE_ERR_INVALID_ARG;
  if (total == 0) return MOE_OK;
  if (slots == nullptr || offsets == nullptr || pos == nullptr || k_new == nullptr || v_new == nullptr ||
      !aligned16(k_new) || !aligned16(v_new))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_cache_write(view_of(cache), cache_ws(cache, workspace), layer, slots, offsets, pos, n, total,
                                        k_new, v_new, k_stride, v_stride, (cudaStream_t)stream));
}

}  // extern "C"
