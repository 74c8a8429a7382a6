// Entry points of the paged-attention operators: argument checks and launches.
#include <cmath>

#include "paged.h"

using namespace fp4moe;

namespace {

constexpr int32_t kMaxRows = 1 << 20, kMaxSeqs = 1 << 16, kMaxHeads = 1024, kMaxPages = 1 << 27, kMaxGroup = 64;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

fp4moe_status check_cache(const fp4moe_kv_cache& c, PagedKv* kv) {
  if (!c.k || !c.v || (c.fp8 != 0 && c.fp8 != 1) || (c.fp8 ? !c.k_scale || !c.v_scale : c.k_scale || c.v_scale))
    return FP4MOE_ERR_INVALID_ARG;
  if ((c.head_dim != 64 && c.head_dim != 128) || c.kv_heads < 1 || c.kv_heads > kMaxHeads || c.pages < 1 ||
      c.pages > kMaxPages || c.page_size < 16 || c.page_size > 128 || (c.page_size & (c.page_size - 1)))
    return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4)) return FP4MOE_ERR_INVALID_ARG;
  const int size = c.fp8 ? 1 : 2;
  for (const int64_t* s : {&c.k_page, &c.v_page}) {  // page, head and token strides
    const int64_t steps[3] = {s == &c.k_page ? c.k_page : c.v_page, s == &c.k_page ? c.k_head : c.v_head,
                              s == &c.k_page ? c.k_token : c.v_token};
    const int32_t n[3] = {c.pages, c.kv_heads, c.page_size};
    for (int i = 0; i < 3; ++i)
      if (steps[i] < (n[i] > 1 ? 1 : 0) || steps[i] >= (int64_t)1 << 38 || steps[i] * size % 16 != 0) return FP4MOE_ERR_INVALID_ARG;
  }
  int shift = 4;
  while (1 << shift < c.page_size) ++shift;
  *kv = PagedKv{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.k_scale, c.v_scale, c.k_page * size,
                c.k_head * size, c.k_token * size, c.v_page * size, c.v_head * size, c.v_token * size, c.pages, shift,
                c.kv_heads};
  return FP4MOE_OK;
}

fp4moe_status check_batch(const fp4moe_kv_batch& b, int page_size, PagedBatch* out) {
  if (!b.lens || (!b.table && b.table_cols != 0)) return FP4MOE_ERR_INVALID_ARG;
  if (b.rows < 0 || b.rows > kMaxRows || b.seqs < 0 || b.seqs > kMaxSeqs || b.table_cols < 0 ||
      (int64_t)b.table_cols * page_size > 1 << 24)
    return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (b.table_ld < b.table_cols || (!b.starts && b.rows != b.seqs) || !aligned(b.starts, 4) || !aligned(b.lens, 4) ||
      !aligned(b.table, 4))
    return FP4MOE_ERR_INVALID_ARG;
  *out = PagedBatch{b.starts, b.lens, b.table, b.table_ld, b.rows, b.seqs, b.table_cols * page_size};
  return FP4MOE_OK;
}

fp4moe_status check_attn(const fp4moe_kv_cache& c, const fp4moe_attn& a, PagedAttn* out) {
  if (!a.q || (a.out ? a.codes || a.code_scales : !a.codes || !a.code_scales)) return FP4MOE_ERR_INVALID_ARG;
  if (a.q_heads < 1 || a.q_heads % c.kv_heads != 0 || a.q_heads / c.kv_heads > kMaxGroup) return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  const int group = a.q_heads / c.kv_heads;
  const float scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  if (a.codes && group * c.head_dim % 128 != 0) return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (a.q_ld < (int64_t)a.q_heads * c.head_dim || a.q_ld % 8 != 0 || a.q_ld >= (int64_t)1 << 38 || a.window < 0 || a.sinks < 0 ||
      !std::isfinite(scale_log2) || a.scale < 0)
    return FP4MOE_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.codes, 16) || !aligned(a.code_scales, 4))
    return FP4MOE_ERR_INVALID_ARG;
  out->out = PagedOut{a.out, a.codes, a.code_scales, a.q_heads * c.head_dim};
  out->q = a.q;
  out->q_ld = a.q_ld;
  out->q_heads = a.q_heads;
  out->group = group;
  out->window = a.window;
  out->sinks = a.sinks;
  out->scale_log2 = scale_log2;
  return FP4MOE_OK;
}

}  // namespace

extern "C" {

fp4moe_status fp4moe_kv_append(const fp4moe_kv_cache* cache, const fp4moe_kv_batch* batch, const fp4moe_append* args,
                               void* stream) {
  if (!cache || !batch || !args) return FP4MOE_ERR_INVALID_ARG;
  const fp4moe_append& x = *args;
  if (!x.k || !x.v || (x.q != nullptr) != (x.q_out != nullptr)) return FP4MOE_ERR_INVALID_ARG;
  KvAppendArgs a{};
  if (fp4moe_status st = check_cache(*cache, &a.kv)) return st;
  if (fp4moe_status st = check_batch(*batch, cache->page_size, &a.batch)) return st;
  const int64_t D = cache->head_dim, kv_cols = cache->kv_heads * D;
  if (x.q_heads < 0 || x.q_heads > kMaxGroup * kMaxHeads || (x.q_heads > 0) != (x.q != nullptr)) return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (x.rope ? x.rope_dim < 16 || x.rope_dim > D || x.rope_dim % 16 != 0 : x.rope_dim != 0) return FP4MOE_ERR_UNSUPPORTED_SHAPE;
  if (x.pairs != 0 && x.pairs != 1) return FP4MOE_ERR_INVALID_ARG;
  for (int64_t ld : {x.q ? x.q_ld : 0, x.q ? x.q_out_ld : 0, x.k_ld, x.v_ld})
    if (ld % 8 != 0 || ld >= (int64_t)1 << 38) return FP4MOE_ERR_INVALID_ARG;
  if (x.k_ld < kv_cols || x.v_ld < kv_cols || (x.q && (x.q_ld < x.q_heads * D || x.q_out_ld < x.q_heads * D)))
    return FP4MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)x.q, (const void*)x.k, (const void*)x.v, (const void*)x.rope, (const void*)x.q_out})
    if (!aligned(p, 16)) return FP4MOE_ERR_INVALID_ARG;
  if (batch->rows == 0 || batch->seqs == 0) return FP4MOE_OK;
  if (fp4moe_status st = check_device()) return st;
  a.q = x.q, a.k = x.k, a.v = x.v, a.q_ld = x.q_ld, a.k_ld = x.k_ld, a.v_ld = x.v_ld, a.q_heads = x.q_heads;
  a.rope = x.rope, a.rope_dim = x.rope_dim, a.pairs = x.pairs, a.q_out = x.q_out, a.q_out_ld = x.q_out_ld;
  a.head_dim = cache->head_dim, a.fp8 = cache->fp8 != 0;
  return cuda_status(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

size_t fp4moe_attn_decode_workspace_size(const fp4moe_kv_cache* cache, int32_t q_heads) {
  if (!cache || (cache->head_dim != 64 && cache->head_dim != 128) || cache->kv_heads < 1 || cache->kv_heads > kMaxHeads ||
      q_heads < 1 || q_heads % cache->kv_heads != 0 || q_heads / cache->kv_heads > kMaxGroup)
    return 0;
  return attn_decode_workspace(cache->head_dim);
}

fp4moe_status fp4moe_attn_decode(const fp4moe_kv_cache* cache, const fp4moe_kv_batch* batch, const fp4moe_attn* attn,
                                 void* ws, size_t ws_bytes, void* stream) {
  if (!cache || !batch || !attn) return FP4MOE_ERR_INVALID_ARG;
  PagedAttn a{};
  if (fp4moe_status st = check_cache(*cache, &a.kv)) return st;
  if (fp4moe_status st = check_batch(*batch, cache->page_size, &a.batch)) return st;
  if (fp4moe_status st = check_attn(*cache, *attn, &a)) return st;
  if (batch->starts || !aligned(ws, 16)) return FP4MOE_ERR_INVALID_ARG;
  if (ws ? ws_bytes < attn_decode_workspace(cache->head_dim) : ws_bytes != 0 || attn_decode_needs_workspace(a, cache->head_dim))
    return FP4MOE_ERR_WORKSPACE;
  if (batch->rows == 0) return FP4MOE_OK;
  if (fp4moe_status st = check_device()) return st;
  return cuda_status(launch_attn_decode(a, cache->head_dim, cache->fp8 != 0, ws, static_cast<cudaStream_t>(stream)));
}

size_t fp4moe_attn_prompt_workspace_size(const fp4moe_kv_cache* cache, int32_t q_heads) {
  return fp4moe_attn_decode_workspace_size(cache, q_heads) ? attn_prompt_workspace(cache->head_dim) : 0;
}

fp4moe_status fp4moe_attn_prompt(const fp4moe_kv_cache* cache, const fp4moe_kv_batch* batch, const fp4moe_attn* attn,
                                 void* ws, size_t ws_bytes, void* stream) {
  return fp4moe_attn_prompt_debug(cache, batch, attn, nullptr, ws, ws_bytes, stream);
}

fp4moe_status fp4moe_attn_prompt_debug(const fp4moe_kv_cache* cache, const fp4moe_kv_batch* batch, const fp4moe_attn* attn,
                                       const fp4moe_debug* dbg, void* ws, size_t ws_bytes, void* stream) {
  if (!cache || !batch || !attn) return FP4MOE_ERR_INVALID_ARG;
  PagedAttn a{};
  if (fp4moe_status st = check_cache(*cache, &a.kv)) return st;
  if (fp4moe_status st = check_batch(*batch, cache->page_size, &a.batch)) return st;
  if (fp4moe_status st = check_attn(*cache, *attn, &a)) return st;
  if (!batch->starts || !aligned(ws, 16)) return FP4MOE_ERR_INVALID_ARG;
  if (ws ? ws_bytes < attn_prompt_workspace(cache->head_dim) : ws_bytes != 0 || attn_prompt_needs_workspace(a))
    return FP4MOE_ERR_WORKSPACE;
  if (batch->rows == 0 || batch->seqs == 0) return FP4MOE_OK;
  if (fp4moe_status st = check_device()) return st;
  const PromptKnobs knobs{dbg && dbg->wait_limit_ns > 0 ? (uint64_t)dbg->wait_limit_ns : 0, dbg && dbg->withhold_first_stage != 0};
  return cuda_status(launch_attn_prompt(a, cache->head_dim, cache->fp8 != 0, ws, knobs, static_cast<cudaStream_t>(stream)));
}

fp4moe_status fp4moe_attn_prompt_status(void* stream, fp4moe_status* st, int64_t* count) {
  if (fp4moe_status e = check_device()) return e;
  int32_t* word = nullptr;
  if (attn_prompt_status_word(&word) != cudaSuccess) return FP4MOE_ERR_CUDA;
  const fp4moe_status e = fp4moe_get_status(word, stream, st, count);
  return e ? e : fp4moe_clear_status(word, stream);
}

}  // extern "C"
