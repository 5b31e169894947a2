// C ABI of the 8-bit paged key/value cache (declared in include/sage_attn.h): argument checks
// and launches on the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sage_attn.h"
#include "args.h"
#include "kv.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return p != nullptr && ((uintptr_t)p & (a - 1)) == 0; }
// an argument that may be left out
bool aligned_or_null(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// SAGE_OK, or what is wrong with the cache itself
int check_cache(const sage_kv_cache* c) {
  if (c == nullptr) return SAGE_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->table, 4) || !aligned(c->lengths, 4) || !aligned(c->refs, 16) || !aligned(c->status, 4))
    return SAGE_ERR_INVALID_ARG;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return SAGE_ERR_UNSUPPORTED;
  if (c->D != 64 && c->D != 128) return SAGE_ERR_UNSUPPORTED;
  if (c->kind != SAGE_KV_INT8 && c->kind != SAGE_KV_E4M3) return SAGE_ERR_UNSUPPORTED;
  if (c->Hkv < 1 || c->Hkv > 32767 || c->n_pages < 1 || c->n_pages > (1 << 28)) return SAGE_ERR_UNSUPPORTED;
  if (c->n_slots < 1 || c->n_slots > sage::kKvMaxSlots || c->max_pages < 1) return SAGE_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page > 0x7fffff00ll) return SAGE_ERR_UNSUPPORTED;  // lengths are int32
  return SAGE_OK;
}
bool attention_shape_ok(int B, int H, int Hkv, int D, int Nq) {
  if (B < 1 || B > sage::kKvMaxBatch || Hkv < 1 || Hkv > 32767 || H < 1 || H % Hkv != 0 || Nq < 1) return false;
  if (D != 64 && D != 128) return false;
  if ((long long)(H / Hkv) * Nq > (1 << 30)) return false;
  return (long long)B * Hkv * sage::kv_attn_ws_layout(1, H, Hkv, D, Nq).tiles <= 0x7fffffffll;
}

}  // namespace

extern "C" {

int sage_attn_kv_append(const sage_kv_cache* cache, const void* K, const void* V, const float* k_shift,
                        const int* slots, const int* pos, const int* n_new, int B, int Nn, void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned_or_null(k_shift, 16) || !aligned_or_null(slots, 4) ||
      !aligned(pos, 4) || !aligned(n_new, 4))
    return SAGE_ERR_INVALID_ARG;
  if (slots == nullptr && B > cache->n_slots) return SAGE_ERR_INVALID_ARG;
  if (B < 1 || B > 65535 || Nn < 1) return SAGE_ERR_UNSUPPORTED;
  return sage::launch_kv_append(*cache, K, V, k_shift, slots, pos, n_new, B, Nn, static_cast<cudaStream_t>(stream));
}

size_t sage_attn_kv_ws_bytes(int B, int H, int Hkv, int D, int Nq) {
  if (!attention_shape_ok(B, H, Hkv, D, Nq)) return 0;
  return sage::kv_attn_ws_layout(B, H, Hkv, D, Nq).total;
}

int sage_attn_kv_attention(const sage_kv_cache* cache, const void* Q, const int* slots, const int* q_len, void* O,
                           float* LSE, void* ws, size_t ws_bytes, int B, int H, int Nq, int causal, float sm_scale,
                           void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4) || !aligned(ws, 16) || !aligned_or_null(slots, 4) ||
      !aligned_or_null(q_len, 4))
    return SAGE_ERR_INVALID_ARG;
  if (!sage::scale_ok(sm_scale)) return SAGE_ERR_INVALID_ARG;
  if (!attention_shape_ok(B, H, cache->Hkv, cache->D, Nq)) return SAGE_ERR_UNSUPPORTED;
  if (slots == nullptr && B > cache->n_slots) return SAGE_ERR_INVALID_ARG;
  if (ws_bytes < sage::kv_attn_ws_layout(B, H, cache->Hkv, cache->D, Nq).total) return SAGE_ERR_INVALID_ARG;
  if (O == Q) return SAGE_ERR_INVALID_ARG;
  return sage::launch_kv_attention(*cache, Q, slots, q_len, O, LSE, ws, B, H, Nq, causal != 0,
                                   sage::resolve_scale(sm_scale, cache->D), static_cast<cudaStream_t>(stream));
}

int sage_attn_selftest_kv_join(const sage_kv_cache* cache, void* O, float* LSE, void* ws, size_t ws_bytes, int B, int H,
                               int Nq, void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!aligned(O, 16) || !aligned(LSE, 4) || !aligned(ws, 16)) return SAGE_ERR_INVALID_ARG;
  if (!attention_shape_ok(B, H, cache->Hkv, cache->D, Nq)) return SAGE_ERR_UNSUPPORTED;
  if (ws_bytes < sage::kv_attn_ws_layout(B, H, cache->Hkv, cache->D, Nq).total) return SAGE_ERR_INVALID_ARG;
  return sage::launch_kv_join(*cache, O, LSE, ws, B, H, Nq, static_cast<cudaStream_t>(stream));
}

int sage_attn_kv_fork(const sage_kv_cache* cache, const int* src, void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!aligned(src, 4)) return SAGE_ERR_INVALID_ARG;
  return sage::launch_kv_fork(*cache, src, static_cast<cudaStream_t>(stream));
}

int sage_attn_kv_extend(const sage_kv_cache* cache, const int* n_new, int* pos, int* cow, void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!aligned(n_new, 4) || !aligned(pos, 4) || !aligned(cow, 4)) return SAGE_ERR_INVALID_ARG;
  // n_new is read after cow is written
  if (n_new == pos || n_new == cow || pos == cow) return SAGE_ERR_INVALID_ARG;
  return sage::launch_kv_extend(*cache, n_new, pos, cow, static_cast<cudaStream_t>(stream));
}

int sage_attn_kv_truncate(const sage_kv_cache* cache, const int* keep, void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!aligned(keep, 4)) return SAGE_ERR_INVALID_ARG;
  return sage::launch_kv_truncate(*cache, keep, static_cast<cudaStream_t>(stream));
}

size_t sage_attn_kv_compact_ws_bytes(int n_pages) {
  if (n_pages < 1 || n_pages > (1 << 28)) return 0;
  return sage::kv_compact_ws_bytes(n_pages);
}

int sage_attn_kv_compact(const sage_kv_cache* cache, const sage_kv_cache* to, void* ws, size_t ws_bytes,
                         void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_cache(to)) return rc;
  if (cache->page != to->page || cache->Hkv != to->Hkv || cache->D != to->D || cache->kind != to->kind ||
      cache->n_slots != to->n_slots || cache->max_pages != to->max_pages)
    return SAGE_ERR_INVALID_ARG;
  // the pools, tables, lengths and refs are read while the others are written
  if (cache->k == to->k || cache->v == to->v || cache->k_scale == to->k_scale || cache->v_scale == to->v_scale ||
      cache->table == to->table || cache->lengths == to->lengths || cache->refs == to->refs)
    return SAGE_ERR_INVALID_ARG;
  if (!aligned(ws, 16) || ws_bytes < sage::kv_compact_ws_bytes(cache->n_pages)) return SAGE_ERR_INVALID_ARG;
  return sage::launch_kv_compact(*cache, *to, ws, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
