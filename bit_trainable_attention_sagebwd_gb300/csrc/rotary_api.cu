// C ABI of rotary positions (declared in include/sage_attn.h): argument checks and the launch on the caller's stream.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/sage_attn.h"
#include "rotary.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return p != nullptr && ((uintptr_t)p & (a - 1)) == 0; }
bool aligned_or_null(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool heads_ok(const sage_heads* x) {
  return x != nullptr && aligned(x->p, 16) && x->batch % 8 == 0 && x->token % 8 == 0 && x->head % 8 == 0;
}
// one that is written: each axis steps over what the smaller ones reach
bool apart(const sage_heads* x, long long B, long long N, long long H, int D) {
  if (!heads_ok(x)) return false;
  long long stride[3] = {B > 1 ? x->batch : 0, N > 1 ? x->token : 0, H > 1 ? x->head : 0}, n[3] = {B, N, H};
  for (int i = 0; i < 2; ++i)  // the smallest stride first
    for (int j = 0; j < 2 - i; ++j)
      if (stride[j] > stride[j + 1]) {
        const long long s = stride[j], m = n[j];
        stride[j] = stride[j + 1], n[j] = n[j + 1];
        stride[j + 1] = s, n[j + 1] = m;
      }
  __int128 reach = D;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (stride[i] < reach) return false;
    reach += (__int128)stride[i] * (n[i] - 1);
  }
  return true;
}
// the output is the input, or begins elsewhere
bool same_or_apart(const sage_heads* in, const sage_heads* out) {
  return in->p != out->p || (in->batch == out->batch && in->token == out->token && in->head == out->head);
}

}  // namespace

extern "C" {

int sage_attn_rotary(const sage_rotary* r, const sage_heads* Q, const sage_heads* Qo, const sage_heads* K,
                     const sage_heads* Ko, const int* positions, const int* start, const int* cu_seqlens, int B, int N,
                     int S, int H, int Hkv, int D, int inverse, void* stream) {
  if (r == nullptr || !aligned(r->turns, 8) || isnan(r->gain) || isinf(r->gain)) return SAGE_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || r->rot < 16 || r->rot > D || r->rot % 16 != 0) return SAGE_ERR_UNSUPPORTED;
  if (B < 1 || N < 1 || (long long)B * N > 0x7fffffffll || H < 1 || H > 32767) return SAGE_ERR_UNSUPPORTED;
  if (K != nullptr && (Hkv < 1 || Hkv > 32767)) return SAGE_ERR_UNSUPPORTED;
  if (!heads_ok(Q) || !apart(Qo, B, N, H, D) || !same_or_apart(Q, Qo)) return SAGE_ERR_INVALID_ARG;
  if ((K == nullptr) != (Ko == nullptr)) return SAGE_ERR_INVALID_ARG;
  if (K != nullptr && (!heads_ok(K) || !apart(Ko, B, N, Hkv, D) || !same_or_apart(K, Ko))) return SAGE_ERR_INVALID_ARG;
  if (K != nullptr && (Qo->p == Ko->p || Qo->p == K->p || Ko->p == Q->p)) return SAGE_ERR_INVALID_ARG;
  if (!aligned_or_null(positions, 4) || !aligned_or_null(start, 4) || !aligned_or_null(cu_seqlens, 4))
    return SAGE_ERR_INVALID_ARG;
  if (positions != nullptr && (start != nullptr || cu_seqlens != nullptr)) return SAGE_ERR_INVALID_ARG;
  if (cu_seqlens != nullptr && B != 1) return SAGE_ERR_INVALID_ARG;
  if (cu_seqlens != nullptr && (S < 1 || S > (1 << 30))) return SAGE_ERR_UNSUPPORTED;
  sage::RotaryParams p;
  p.r = *r;
  p.in[0] = *Q, p.out[0] = *Qo, p.heads[0] = H;
  p.in[1] = K != nullptr ? *K : *Q, p.out[1] = Ko != nullptr ? *Ko : *Qo, p.heads[1] = K != nullptr ? Hkv : 0;
  p.positions = positions, p.start = start, p.cu = cu_seqlens;
  p.B = B, p.N = N, p.S = S, p.inverse = inverse != 0;
  return sage::launch_rotary(p, D, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
