// C ABI of attention over packed sequences (declared in include/sage_attn.h): argument checks and launches on the
// caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sage_attn.h"
#include "args.h"
#include "packed.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return p != nullptr && ((uintptr_t)p & (a - 1)) == 0; }

bool shape_ok(int T, int S, int H, int Hkv, int D) {
  if (T < 1 || T > sage::kPackedMaxTokens || S < 1 || S > sage::kPackedMaxSeqs) return false;
  if (Hkv < 1 || H < 1 || H > 32767 || H % Hkv != 0 || H / Hkv > sage::kPackedMaxGroup) return false;
  return D == 64 || D == 128;
}

// A tensor [T, heads, D]: rows of 16-byte pieces, the strides such that TMA takes them (below 2^40 bytes)
bool rows_ok(const sage_rows* x, int T, int heads) {
  if (x == nullptr || !aligned(x->p, 16)) return false;
  const long long most = 1ll << 38;
  auto ok = [&](long long stride, int n) { return n == 1 || (stride > 0 && stride < most && stride % 8 == 0); };
  return ok(x->token, T) && ok(x->head, heads);
}
// one that is written: its rows lie apart
bool apart(const sage_rows* x, int T, int heads, int D) {
  if (!rows_ok(x, T, heads)) return false;
  const long long token = T == 1 ? 0 : x->token, head = heads == 1 ? 0 : x->head;
  if (T == 1 || heads == 1) return T == 1 && heads == 1 ? true : (T == 1 ? head : token) >= D;
  return head < token ? head >= D && token >= head * (heads - 1) + D : token >= D && head >= token * (T - 1) + D;
}

}  // namespace

extern "C" {

size_t sage_attn_packed_ws_bytes(int T, int S, int H, int Hkv, int D, int backward) {
  if (!shape_ok(T, S, H, Hkv, D)) return 0;
  return sage::packed_ws_layout(T, S, H, Hkv, D, backward != 0).total;
}

int sage_attn_packed_fwd(const sage_rows* Q, const sage_rows* K, const sage_rows* V, const int* cu_seqlens,
                         const sage_rows* O, float* LSE, void* ws, size_t ws_bytes, int T, int S, int H, int Hkv, int D,
                         int causal, float sm_scale, void* stream) {
  if (!shape_ok(T, S, H, Hkv, D)) return SAGE_ERR_UNSUPPORTED;
  if (!rows_ok(Q, T, H) || !rows_ok(K, T, Hkv) || !rows_ok(V, T, Hkv) || !apart(O, T, H, D)) return SAGE_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 4) || !aligned(LSE, 4) || !aligned(ws, 256) || !sage::scale_ok(sm_scale)) return SAGE_ERR_INVALID_ARG;
  if (ws_bytes < sage::packed_ws_layout(T, S, H, Hkv, D, false).total) return SAGE_ERR_INVALID_ARG;
  if (O->p == Q->p || O->p == K->p || O->p == V->p) return SAGE_ERR_INVALID_ARG;
  return sage::launch_packed_fwd(*Q, *K, *V, cu_seqlens, *O, LSE, ws, T, S, H, Hkv, D, causal != 0,
                                 sage::resolve_scale(sm_scale, D), static_cast<cudaStream_t>(stream));
}

int sage_attn_packed_bwd(const sage_rows* Q, const sage_rows* K, const sage_rows* V, const sage_rows* O, const float* LSE,
                         const sage_rows* dO, const int* cu_seqlens, const sage_rows* dQ, const sage_rows* dK,
                         const sage_rows* dV, void* ws, size_t ws_bytes, int T, int S, int H, int Hkv, int D, int causal,
                         float sm_scale, void* stream) {
  if (!shape_ok(T, S, H, Hkv, D) || (sm_scale > 0.f && sm_scale < sage::kPackedLeastScale)) return SAGE_ERR_UNSUPPORTED;
  if (!rows_ok(Q, T, H) || !rows_ok(K, T, Hkv) || !rows_ok(V, T, Hkv) || !rows_ok(O, T, H) || !rows_ok(dO, T, H) ||
      !apart(dQ, T, H, D) || !apart(dK, T, Hkv, D) || !apart(dV, T, Hkv, D))
    return SAGE_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 4) || !aligned(LSE, 4) || !aligned(ws, 256) || !sage::scale_ok(sm_scale)) return SAGE_ERR_INVALID_ARG;
  if (ws_bytes < sage::packed_ws_layout(T, S, H, Hkv, D, true).total) return SAGE_ERR_INVALID_ARG;
  const void* read[] = {Q->p, K->p, V->p, O->p, dO->p, LSE};
  const void* written[] = {dQ->p, dK->p, dV->p};
  for (const void* w : written)
    for (const void* r : read)
      if (w == r) return SAGE_ERR_INVALID_ARG;
  if (dQ->p == dK->p || dQ->p == dV->p || dK->p == dV->p) return SAGE_ERR_INVALID_ARG;
  return sage::launch_packed_bwd(*Q, *K, *V, *O, LSE, *dO, cu_seqlens, *dQ, *dK, *dV, ws, T, S, H, Hkv, D, causal != 0,
                                 sage::resolve_scale(sm_scale, D), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
