// Host side of attention over key ranges: argument checks, tensor maps, the
// entry points.
#include <algorithm>

#include "attn_ops.h"
#include "tensor_map.h"

namespace httm {
namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 38;       // elements: TMA strides stay below 2^40 bytes

// Extents, types and limits; pointers come later.
httm_status check_attention(const httm_attention* a) {
  if (!a) return HTTM_ERR_ARG;
  if (a->batch < 0 || a->q_len < 0 || a->kv_len < 0 || a->heads < 1 || a->kv_heads < 1) return HTTM_ERR_ARG;
  if (a->heads % a->kv_heads != 0 || a->d_head < 1) return HTTM_ERR_ARG;
  if (a->dtype != HTTM_BF16 && a->dtype != HTTM_F32) return HTTM_ERR_ARG;
  // 0 or within 2^-64 .. 2^64 (lse / scale has to stay finite)
  if (!(a->softmax_scale == 0.f || (a->softmax_scale >= 0x1p-64f && a->softmax_scale <= 0x1p64f))) return HTTM_ERR_ARG;
  if (a->dtype != HTTM_BF16 || a->d_head % 8 != 0 || a->d_head > kAttnD) return HTTM_ERR_UNSUPPORTED;
  if (a->q_len > kAttnMaxQ || a->kv_len > (1 << 30)) return HTTM_ERR_UNSUPPORTED;
  const long long G = a->heads / a->kv_heads;
  const long long bh = (long long)a->batch * a->heads;
  if (bh > 65535 || G * a->q_len > (1ll << 30)) return HTTM_ERR_UNSUPPORTED;
  // every grid and padded row count fits in 31 bits
  const long long q_tiles = (a->q_len + kAttnTile - 1) / kAttnTile, k_tiles = (a->kv_len + kAttnTile - 1) / kAttnTile;
  if (bh * q_tiles > 0x7ffffffll || (long long)a->batch * a->kv_heads * k_tiles > 0x7ffffffll)
    return HTTM_ERR_UNSUPPORTED;
  return HTTM_OK;
}

// One tensor argument with extents (batch, heads, tokens, d).
httm_status check_view(const httm_view* v, int64_t batch, int64_t heads, int64_t tokens, int d, bool output,
                       View* out) {
  *out = View{nullptr, 0, 0, 0};
  if (!v) return HTTM_ERR_ARG;
  if (batch == 0 || tokens == 0) return HTTM_OK;
  if (!v->data) return HTTM_ERR_ARG;
  const View w = normal_view(*v, batch, heads, tokens);
  for (int64_t s : {w.sb, w.sh, w.st})
    if (s < 0 || s >= kMaxStride) return HTTM_ERR_ARG;
  if (!aligned(w.data, 16) || w.sb % 8 || w.sh % 8 || w.st % 8) return HTTM_ERR_ALIGN;
  if (tokens > 1 && w.st == 0) return HTTM_ERR_ARG;
  if (output && !disjoint(w, batch, heads, tokens, d)) return HTTM_ERR_ARG;
  *out = w;
  return HTTM_OK;
}

AttnArgs base_args(const httm_attention& a) {
  AttnArgs g{};
  g.B = a.batch, g.H = a.heads, g.K = a.kv_heads, g.G = a.heads / a.kv_heads, g.L = a.q_len, g.N = a.kv_len;
  g.d = a.d_head;
  g.scale = a.softmax_scale > 0.f ? a.softmax_scale : 1.f / sqrtf((float)a.d_head);
  g.scale_log2 = g.scale * 1.4426950408889634f;
  g.kb = a.key_begin;
  g.ke = a.key_end;
  return g;
}

}  // namespace

bool attn_map(AttnMap* m, const View& v, const void* spare, int d, int tokens, int heads, int batch, int rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  m->hmul = heads > 1 && v.sh > 0 ? 1 : 0;
  m->bmul = batch > 1 && v.sb > 0 ? 1 : 0;
  const void* base = v.data ? v.data : spare;
  const cuuint64_t row = (cuuint64_t)d * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)std::max(1, tokens), (cuuint64_t)(m->hmul ? heads : 1),
                              (cuuint64_t)(m->bmul ? batch : 1)};
  const cuuint64_t strides[3] = {tokens > 1 ? (cuuint64_t)v.st * 2 : row, m->hmul ? (cuuint64_t)v.sh * 2 : row,
                                 m->bmul ? (cuuint64_t)v.sb * 2 : row};
  const cuuint32_t box[4] = {(cuuint32_t)kAttnD, (cuuint32_t)rows, 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return enc(&m->map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace httm

using namespace httm;

extern "C" {

httm_status httm_attention_workspace_bytes(const httm_attention* a, size_t* forward, size_t* backward) {
  HTTM_TRY(check_attention(a));
  const bool none = a->batch == 0;
  // enough for calls with key ranges and without
  if (forward)
    *forward = none || a->q_len == 0
                   ? 0 : std::max(attn_fwd_plan(*a, true).part_bytes, attn_fwd_plan(*a, false).part_bytes);
  if (backward) *backward = none ? 0 : attn_bwd_plan(*a).total;
  return HTTM_OK;
}

httm_status httm_attention_forward(const httm_attention* a, const httm_view* q, const httm_view* k,
                                   const httm_view* v, const httm_view* out, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  HTTM_TRY(check_attention(a));
  AttnArgs g = base_args(*a);
  HTTM_TRY(check_view(q, g.B, g.H, g.L, g.d, false, &g.q));
  HTTM_TRY(check_view(k, g.B, g.K, g.N, g.d, false, &g.k));
  HTTM_TRY(check_view(v, g.B, g.K, g.N, g.d, false, &g.v));
  HTTM_TRY(check_view(out, g.B, g.H, g.L, g.d, true, &g.out));
  if (!aligned(lse, 4) || !aligned(g.kb, 4) || !aligned(g.ke, 4)) return HTTM_ERR_ALIGN;
  if (g.B == 0 || g.L == 0) return HTTM_OK;
  const AttnFwdPlan p = attn_fwd_plan(*a, a->key_begin || a->key_end);
  if (p.part_bytes && (!workspace || workspace_bytes < p.part_bytes)) return HTTM_ERR_WORKSPACE;
  if (p.part_bytes && !aligned(workspace, 256)) return HTTM_ERR_ALIGN;
  g.lse = lse;
  g.st = ops_state();
  if (!g.st) return cuda_fail(cudaGetLastError(), "ops_state");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  HTTM_OPS_LAUNCH(launch_attn_fwd(g, p, workspace, s), s);
  return HTTM_OK;
}

httm_status httm_attention_backward(const httm_attention* a, const httm_view* dout, const httm_view* q,
                                    const httm_view* k, const httm_view* v, const httm_view* out, const float* lse,
                                    const httm_view* dq, const httm_view* dk, const httm_view* dv, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  HTTM_TRY(check_attention(a));
  AttnArgs g = base_args(*a);
  HTTM_TRY(check_view(dout, g.B, g.H, g.L, g.d, false, &g.dout));
  HTTM_TRY(check_view(q, g.B, g.H, g.L, g.d, false, &g.q));
  HTTM_TRY(check_view(k, g.B, g.K, g.N, g.d, false, &g.k));
  HTTM_TRY(check_view(v, g.B, g.K, g.N, g.d, false, &g.v));
  HTTM_TRY(check_view(out, g.B, g.H, g.L, g.d, false, &g.out));
  HTTM_TRY(check_view(dq, g.B, g.H, g.L, g.d, true, &g.dq));
  HTTM_TRY(check_view(dk, g.B, g.K, g.N, g.d, true, &g.dk));
  HTTM_TRY(check_view(dv, g.B, g.K, g.N, g.d, true, &g.dv));
  if (g.B > 0 && g.L > 0 && !lse) return HTTM_ERR_ARG;
  if (!aligned(lse, 4) || !aligned(g.kb, 4) || !aligned(g.ke, 4)) return HTTM_ERR_ALIGN;
  if (g.B == 0 || (g.L == 0 && g.N == 0)) return HTTM_OK;
  const AttnBwdPlan p = attn_bwd_plan(*a);
  if (p.total && (!workspace || workspace_bytes < p.total)) return HTTM_ERR_WORKSPACE;
  if (p.total && !aligned(workspace, 256)) return HTTM_ERR_ALIGN;
  g.lse_in = lse;
  g.st = ops_state();
  if (!g.st) return cuda_fail(cudaGetLastError(), "ops_state");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  HTTM_OPS_LAUNCH(launch_attn_bwd(g, p, workspace, s), s);
  return HTTM_OK;
}

}  // extern "C"
