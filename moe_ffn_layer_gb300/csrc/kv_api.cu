// C ABI of the 8-bit paged KV cache: argument checks and launches.
#include <limits.h>

#include "common.cuh"
#include "kernels.h"

namespace {

inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_dims(const moe_kv_dims* d) {
  if (!d || d->Hkv <= 0 || d->D <= 0 || d->page <= 0) return MOE_ERR_INVALID;
  if ((d->D != 64 && d->D != 128) || d->Hkv > 32767) return MOE_ERR_UNSUPPORTED;
  if (d->page != 16 && d->page != 32 && d->page != 64 && d->page != 128) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_seqs(const moe_kv_seqs* s) {
  if (!s || s->B < 0 || s->width < 0 || s->max_len < 0) return MOE_ERR_INVALID;
  // (a grid's z; positions a few tiles past the end still fit an int)
  if (s->B > 65535 || s->max_len > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// what a call with work to do needs of its pool and sequences
int check_pointers(const moe_kv_dims* d, const moe_kv_pool* p, const moe_kv_seqs* s) {
  // (the rows of a pool are counted in 32 bits: 2^32 of 64 bytes pass the card's memory with K and V)
  if (static_cast<uint64_t>(p->num_pages) * d->Hkv * d->page > UINT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (!s->seq_lens || (s->width > 0 && !s->page_table)) return MOE_ERR_INVALID;
  if (p->num_pages > 0 && (!p->k || !p->v || !p->k_scale || !p->v_scale)) return MOE_ERR_INVALID;
  if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->k_scale, 4) || !aligned(p->v_scale, 4) ||
      !aligned(s->page_table, 4) || !aligned(s->seq_lens, 4))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe::KvDims dims_of(const moe_kv_dims* d) { return {d->Hkv, d->D, d->page, __builtin_ctz(d->page)}; }
moe::KvPool pool_of(const moe_kv_pool* p) {
  return {static_cast<uint8_t*>(p->k), static_cast<uint8_t*>(p->v), p->k_scale, p->v_scale, p->num_pages};
}
moe::KvSeqs seqs_of(const moe_kv_seqs* s) { return {s->page_table, s->seq_lens, s->B, s->width, s->max_len}; }

}  // namespace

extern "C" {

int moe_kv_append(const moe_kv_dims* d, const moe_kv_pool* pool, const moe_kv_seqs* s, const void* k, const void* v,
                  int64_t kv_stride, const int32_t* cu_new, int T_new, cudaStream_t stream) {
  moe::set_last_launches(0);
  int rc = check_dims(d);
  if (rc || (rc = check_seqs(s))) return rc;
  if (!pool || pool->num_pages < 0 || T_new < 0) return MOE_ERR_INVALID;
  if (kv_stride < static_cast<int64_t>(d->Hkv) * d->D) return MOE_ERR_INVALID;
  if (kv_stride % 8) return MOE_ERR_UNSUPPORTED;
  if (T_new == 0 || s->B == 0) return MOE_OK;
  if (!k || !v || !cu_new) return MOE_ERR_INVALID;
  if ((rc = check_pointers(d, pool, s))) return rc;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu_new, 4)) return MOE_ERR_UNSUPPORTED;
  int* status = nullptr;
  int sms = 0, n = 0;
  if ((rc = moe::current_device_info(&status, &sms))) return rc;
  rc = moe::kv_append_launch(dims_of(d), pool_of(pool), seqs_of(s), k, v, kv_stride, cu_new, T_new, status, stream, &n);
  moe::set_last_launches(n);
  return rc;
}

size_t moe_kv_attention_workspace_bytes(const moe_kv_dims* d, int Hq, int B, int T_q, int max_q, int max_len,
                                        int weights) {
  if (check_dims(d) || Hq <= 0 || Hq % d->Hkv || B < 0 || T_q < 0 || max_q < 0 || max_len < 0) return 0;
  return moe::kv_attention_ws_bytes(dims_of(d), Hq, B, T_q, max_q, max_len, weights != 0);
}

int moe_kv_attention(const moe_kv_dims* d, const moe_kv_pool* pool, const moe_kv_seqs* s, const void* q,
                     int64_t q_stride, int Hq, const int32_t* cu_q, int T_q, int max_q, float scale, void* out,
                     float* lse, float* weights, int64_t w_stride, void* ws, size_t ws_bytes, cudaStream_t stream) {
  moe::set_last_launches(0);
  int rc = check_dims(d);
  if (rc || (rc = check_seqs(s))) return rc;
  if (!pool || pool->num_pages < 0 || Hq <= 0 || Hq % d->Hkv || T_q < 0 || max_q < 0) return MOE_ERR_INVALID;
  if (q_stride < static_cast<int64_t>(Hq) * d->D || (weights && w_stride < s->max_len)) return MOE_ERR_INVALID;
  if (q_stride % 8 || static_cast<int64_t>(max_q) * Hq > INT_MAX) return MOE_ERR_UNSUPPORTED;
  if (T_q == 0 || max_q == 0 || s->B == 0) return MOE_OK;
  if (!q || !cu_q || !out || !ws) return MOE_ERR_INVALID;
  if ((rc = check_pointers(d, pool, s))) return rc;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cu_q, 4) || !aligned(lse, 4) || !aligned(weights, 4) ||
      !aligned(ws, 256))
    return MOE_ERR_UNSUPPORTED;
  const moe::KvDims kd = dims_of(d);
  if (ws_bytes < moe::kv_attention_ws_bytes(kd, Hq, s->B, T_q, max_q, s->max_len, weights != nullptr))
    return MOE_ERR_WORKSPACE;
  int* status = nullptr;
  int sms = 0, n = 0;
  if ((rc = moe::current_device_info(&status, &sms))) return rc;
  const moe::KvAttention a{q, q_stride, Hq, cu_q, T_q, max_q, scale, out, lse, weights, w_stride, 0};
  rc = moe::kv_attention_launch(kd, pool_of(pool), seqs_of(s), a, ws, status, stream, &n);
  moe::set_last_launches(n);
  return rc;
}

int moe_kv_evict(const moe_kv_dims* d, const moe_kv_pool* src, const moe_kv_seqs* s, const float* weights,
                 int64_t w_stride, int budget, int sink, int recent, const moe_kv_pool* dst, const int32_t* dst_table,
                 int dst_width, int32_t* dst_lens, float* dst_weights, int32_t* kept, cudaStream_t stream) {
  moe::set_last_launches(0);
  int rc = check_dims(d);
  if (rc || (rc = check_seqs(s))) return rc;
  if (!src || src->num_pages < 0 || !dst || dst->num_pages < 0 || dst_width < 0) return MOE_ERR_INVALID;
  if (budget <= 0 || sink < 0 || recent < 0 || sink > budget - recent || w_stride < s->max_len) return MOE_ERR_INVALID;
  const int most = s->max_len < budget ? s->max_len : budget;
  if (static_cast<int64_t>(dst_width) * d->page < most) return MOE_ERR_INVALID;
  if (s->B == 0) return MOE_OK;
  if (!weights || !dst_lens || !dst_weights || !kept || (dst_width > 0 && !dst_table)) return MOE_ERR_INVALID;
  if ((rc = check_pointers(d, src, s)) || (rc = check_pointers(d, dst, s))) return rc;
  if (!aligned(weights, 4) || !aligned(dst_table, 4) || !aligned(dst_lens, 4) || !aligned(dst_weights, 4) ||
      !aligned(kept, 4))
    return MOE_ERR_UNSUPPORTED;
  int* status = nullptr;
  int sms = 0, n = 0;
  if ((rc = moe::current_device_info(&status, &sms))) return rc;
  const moe::KvEvict e{weights, w_stride, budget, sink, recent, dst_table, dst_width, dst_lens, dst_weights, kept};
  rc = moe::kv_evict_launch(dims_of(d), pool_of(src), seqs_of(s), pool_of(dst), e, status, stream, &n);
  moe::set_last_launches(n);
  return rc;
}

}  // extern "C"
