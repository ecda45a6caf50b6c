// Host layer of the attention block: argument checks and launches.  Every check runs before
// anything is enqueued; nothing here allocates or synchronises.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "attn_kernels.hpp"

using namespace lora;

namespace {

constexpr int MAX_TOKENS = 65536;
constexpr int MAX_HEADS = 1024;
constexpr int MAX_DRAFT_WORDS = 16;

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

lora_status check_heads(int32_t T, int32_t n_q, int32_t n_kv, int32_t D) {
  if (T < 0 || n_q < 1 || n_kv < 1 || D < 1) return LORA_ERR_INVALID_ARG;
  if (T > MAX_TOKENS || n_q > MAX_HEADS || n_kv > MAX_HEADS) return LORA_ERR_UNSUPPORTED;
  return D == 64 || D == 128 || D == 256 ? LORA_OK : LORA_ERR_UNSUPPORTED;
}

// A row-major matrix of bf16 rows read and written in 16-byte pieces.
inline bool rows_ok(const void* p, int64_t ld, int64_t width) { return p && aligned(p, 16) && ld >= width && ld % 8 == 0; }

lora_status check_rope(const int32_t* positions, const float* cos_sin, int32_t max_pos, int32_t rot, int32_t D,
                       int32_t interleaved, const float* qw, const float* kw, float eps) {
  if (rot < 0 || rot > D || (interleaved != 0 && interleaved != 1)) return LORA_ERR_INVALID_ARG;
  if (rot % 16 != 0) return LORA_ERR_UNSUPPORTED;
  if (rot > 0 && (!positions || !aligned(positions, 4) || !cos_sin || !aligned(cos_sin, 16) || max_pos < 1))
    return LORA_ERR_INVALID_ARG;
  if ((qw == nullptr) != (kw == nullptr)) return LORA_ERR_INVALID_ARG;
  if (qw && (!aligned(qw, 16) || !aligned(kw, 16) || !(eps >= 0.f) || !isfinite(eps))) return LORA_ERR_INVALID_ARG;
  return LORA_OK;
}

// How a call gives its tokens' positions: one each (n 0), or on n axes, with an axis for each pair.
struct Axes { int32_t n; const uint8_t* of_pair; };

lora_status axis_map(const Axes& by, int32_t rot, AxisMap* m) {
  m->n = by.n;
  if (by.n == 0) return LORA_OK;
  if (rot > 0 && !by.of_pair) return LORA_ERR_INVALID_ARG;
  m->quads = 1;
  for (int32_t i = 0; i < rot / 2; ++i) {
    const uint64_t axis = by.of_pair[i];
    if (axis >= (uint64_t)by.n) return LORA_ERR_INVALID_ARG;
    m->pair[i / 32] |= axis << (2 * (i % 32));
    if (i % 4 == 0) m->quad |= axis << (i / 2);
    else if (axis != by.of_pair[i / 4 * 4]) m->quads = 0;
  }
  return LORA_OK;
}

// Calls that take axes take one at least, and four at most.
inline lora_status check_axes(int32_t n) {
  return n < 1 ? LORA_ERR_INVALID_ARG : n > 4 ? LORA_ERR_UNSUPPORTED : LORA_OK;
}

lora_status check_pages(int32_t n_pages, int32_t page_size, int32_t n_kv, int32_t* log2_out) {
  if (n_pages < 1 || page_size < 1) return LORA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1))) return LORA_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * page_size > INT32_MAX) return LORA_ERR_UNSUPPORTED;
  int l = 4;
  while ((1 << l) < page_size) ++l;
  *log2_out = l;
  return LORA_OK;
}

inline bool cache_fmt_ok(int32_t fmt) { return fmt == LORA_KV_BF16 || fmt == LORA_KV_FP8_E4M3; }

RopeParams rope_params(const uint16_t* qkv, int64_t ld, const int32_t* positions, int32_t T, int32_t n_q, int32_t n_kv,
                       const float* cos_sin, int32_t max_pos, int32_t rot, int32_t interleaved, const float* qw,
                       const float* kw, float eps, uint16_t* q_out, int64_t ldq, int32_t* status) {
  RopeParams p{};
  p.qkv = qkv; p.ld = ld; p.positions = positions; p.T = T; p.n_q = n_q; p.n_kv = n_kv;
  p.cos_sin = cos_sin; p.max_pos = max_pos; p.rot = rot; p.interleaved = interleaved;
  p.q_weight = qw; p.k_weight = kw; p.eps = eps; p.q_out = q_out; p.ldq = ldq; p.status = status;
  return p;
}

inline size_t plan_bytes(const TreeAttnPlan& pl) {
  return round256(pl.desc_bytes) + round256(pl.ml_bytes) + round256(pl.o_bytes);
}

lora_status norm_rope(const uint16_t* qkv, int64_t ld, const int32_t* positions, const Axes& by, int32_t T,
                      int32_t n_q, int32_t n_kv, int32_t D, const float* cos_sin, int32_t max_pos, int32_t rot,
                      int32_t interleaved, const float* q_weight, const float* k_weight, float eps, uint16_t* q_out,
                      int64_t ldq, uint16_t* k_out, int64_t ldk, int32_t* status, void* stream) {
  AxisMap axes{};
  lora_status st = check_heads(T, n_q, n_kv, D);
  if (st != LORA_OK) return st;
  st = check_rope(positions, cos_sin, max_pos, rot, D, interleaved, q_weight, k_weight, eps);
  if (T == 0 && st != LORA_ERR_UNSUPPORTED) return LORA_OK;
  if (st != LORA_OK || (st = axis_map(by, rot, &axes)) != LORA_OK) return st;
  if (!rows_ok(qkv, ld, (int64_t)(n_q + 2 * n_kv) * D) || !rows_ok(q_out, ldq, (int64_t)n_q * D) ||
      !rows_ok(k_out, ldk, (int64_t)n_kv * D) || !aligned(status, 4))
    return LORA_ERR_INVALID_ARG;
  RopeParams p = rope_params(qkv, ld, positions, T, n_q, n_kv, cos_sin, max_pos, rot, interleaved, q_weight, k_weight,
                             eps, q_out, ldq, status);
  p.k_out = k_out; p.ldk = ldk; p.axes = axes;
  return launch_norm_rope(p, D, as_stream(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status rope_append(const uint16_t* qkv, int64_t ld, const int32_t* positions, const Axes& by,
                        const int32_t* slots, int32_t T, int32_t n_q, int32_t n_kv, int32_t D, const float* cos_sin,
                        int32_t max_pos, int32_t rot, int32_t interleaved, const float* q_weight,
                        const float* k_weight, float eps, uint16_t* q_out, int64_t ldq, int32_t kv_fmt, void* k_cache,
                        void* v_cache, const float* k_scale, const float* v_scale, int32_t n_pages, int32_t page_size,
                        int32_t* status, void* stream) {
  AxisMap axes{};
  lora_status st = check_heads(T, n_q, n_kv, D);
  if (st != LORA_OK) return st;
  int32_t lg = 0;
  if (!cache_fmt_ok(kv_fmt)) return LORA_ERR_INVALID_ARG;
  if ((st = check_pages(n_pages, page_size, n_kv, &lg)) != LORA_OK) return st;
  st = check_rope(positions, cos_sin, max_pos, rot, D, interleaved, q_weight, k_weight, eps);
  if (T == 0 && st != LORA_ERR_UNSUPPORTED) return LORA_OK;
  if (st != LORA_OK || (st = axis_map(by, rot, &axes)) != LORA_OK) return st;
  if (!rows_ok(qkv, ld, (int64_t)(n_q + 2 * n_kv) * D) || !rows_ok(q_out, ldq, (int64_t)n_q * D) || !slots ||
      !aligned(slots, 4) || !k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(status, 4))
    return LORA_ERR_INVALID_ARG;
  const bool fp8 = kv_fmt == LORA_KV_FP8_E4M3;
  if (fp8 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4))) return LORA_ERR_INVALID_ARG;
  RopeParams p = rope_params(qkv, ld, positions, T, n_q, n_kv, cos_sin, max_pos, rot, interleaved, q_weight, k_weight,
                             eps, q_out, ldq, status);
  p.slots = slots; p.k_cache = k_cache; p.v_cache = v_cache; p.k_scale = k_scale; p.v_scale = v_scale;
  p.page_log2 = lg; p.n_slots = (long)n_pages * page_size;
  p.axes = axes;
  return launch_rope_append(p, D, fp8, as_stream(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

size_t rope_backward_workspace(int32_t T, int32_t D) {
  if (T < 1 || T > MAX_TOKENS || (D != 64 && D != 128 && D != 256)) return 0;
  return (size_t)ROPE_BWD_WGS * D * sizeof(float);
}

lora_status norm_rope_backward(const uint16_t* qkv, int64_t ld, const int32_t* positions, const Axes& by,
                               const uint16_t* dq, const uint16_t* dk, const uint16_t* dv, int32_t T, int32_t n_q,
                               int32_t n_kv, int32_t D, const float* cos_sin, int32_t max_pos, int32_t rot,
                               int32_t interleaved, const float* q_weight, const float* k_weight, float eps,
                               uint16_t* dqkv, int64_t ldd, float* dq_weight, float* dk_weight, int32_t* status,
                               void* workspace, size_t workspace_bytes, void* stream) {
  AxisMap axes{};
  lora_status st = check_heads(T, n_q, n_kv, D);
  if (st != LORA_OK) return st;
  st = check_rope(positions, cos_sin, max_pos, rot, D, interleaved, q_weight, k_weight, eps);
  if (st == LORA_ERR_UNSUPPORTED || (st != LORA_OK && T > 0)) return st;
  if (T > 0 && (st = axis_map(by, rot, &axes)) != LORA_OK) return st;
  const bool norm = q_weight != nullptr;
  if (norm && (!dq_weight || !dk_weight || !aligned(dq_weight, 16) || !aligned(dk_weight, 16))) return LORA_ERR_INVALID_ARG;
  RopeBwdParams p{};
  p.T = T; p.dqw = dq_weight; p.dkw = dk_weight; p.q_weight = q_weight; p.k_weight = k_weight;
  if (T > 0) {
    const int64_t width = (int64_t)(n_q + 2 * n_kv) * D;
    if (!rows_ok(dqkv, ldd, width) || !dq || !dk || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
        !aligned(status, 4) || (norm && !rows_ok(qkv, ld, width)))
      return LORA_ERR_INVALID_ARG;
    const size_t need = norm ? rope_backward_workspace(T, D) : 0;
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return LORA_ERR_WORKSPACE;
  }
  p.qkv = qkv; p.ld = ld; p.positions = positions; p.n_q = n_q; p.n_kv = n_kv;
  p.cos_sin = cos_sin; p.max_pos = max_pos; p.rot = rot; p.interleaved = interleaved; p.eps = eps;
  p.dq = dq; p.dk = dk; p.dv = dv; p.dqkv = dqkv; p.ldd = ldd;
  p.part = reinterpret_cast<float*>(workspace); p.status = status;
  p.axes = axes;
  return launch_norm_rope_bwd(p, D, as_stream(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // namespace

extern "C" {

lora_status lora_qk_norm_rope(const uint16_t* qkv, int64_t ld, const int32_t* positions, int32_t T, int32_t n_q,
                              int32_t n_kv, int32_t D, const float* cos_sin, int32_t max_pos, int32_t rot,
                              int32_t interleaved, const float* q_weight, const float* k_weight, float eps,
                              uint16_t* q_out, int64_t ldq, uint16_t* k_out, int64_t ldk, int32_t* status,
                              void* stream) {
  return norm_rope(qkv, ld, positions, {0, nullptr}, T, n_q, n_kv, D, cos_sin, max_pos, rot, interleaved, q_weight,
                   k_weight, eps, q_out, ldq, k_out, ldk, status, stream);
}

lora_status lora_qk_norm_rope_axes(const uint16_t* qkv, int64_t ld, const int32_t* positions, int32_t n_axes,
                                   const uint8_t* pair_axes, int32_t T, int32_t n_q, int32_t n_kv, int32_t D,
                                   const float* cos_sin, int32_t max_pos, int32_t rot, int32_t interleaved,
                                   const float* q_weight, const float* k_weight, float eps, uint16_t* q_out, int64_t ldq,
                                   uint16_t* k_out, int64_t ldk, int32_t* status, void* stream) {
  const lora_status st = check_axes(n_axes);
  if (st != LORA_OK) return st;
  return norm_rope(qkv, ld, positions, {n_axes, pair_axes}, T, n_q, n_kv, D, cos_sin, max_pos, rot, interleaved,
                   q_weight, k_weight, eps, q_out, ldq, k_out, ldk, status, stream);
}

lora_status lora_rope_append_kv(const uint16_t* qkv, int64_t ld, const int32_t* positions, const int32_t* slots,
                                int32_t T, int32_t n_q, int32_t n_kv, int32_t D, const float* cos_sin, int32_t max_pos,
                                int32_t rot, int32_t interleaved, const float* q_weight, const float* k_weight,
                                float eps, uint16_t* q_out, int64_t ldq, int32_t kv_fmt, void* k_cache, void* v_cache,
                                const float* k_scale, const float* v_scale, int32_t n_pages, int32_t page_size,
                                int32_t* status, void* stream) {
  return rope_append(qkv, ld, positions, {0, nullptr}, slots, T, n_q, n_kv, D, cos_sin, max_pos, rot, interleaved,
                     q_weight, k_weight, eps, q_out, ldq, kv_fmt, k_cache, v_cache, k_scale, v_scale, n_pages,
                     page_size, status, stream);
}

lora_status lora_rope_axes_append_kv(const uint16_t* qkv, int64_t ld, const int32_t* positions, int32_t n_axes,
                                     const uint8_t* pair_axes, const int32_t* slots, int32_t T, int32_t n_q,
                                     int32_t n_kv, int32_t D, const float* cos_sin, int32_t max_pos, int32_t rot,
                                     int32_t interleaved, const float* q_weight, const float* k_weight, float eps,
                                     uint16_t* q_out, int64_t ldq, int32_t kv_fmt, void* k_cache, void* v_cache,
                                     const float* k_scale, const float* v_scale, int32_t n_pages, int32_t page_size,
                                     int32_t* status, void* stream) {
  const lora_status st = check_axes(n_axes);
  if (st != LORA_OK) return st;
  return rope_append(qkv, ld, positions, {n_axes, pair_axes}, slots, T, n_q, n_kv, D, cos_sin, max_pos, rot,
                     interleaved, q_weight, k_weight, eps, q_out, ldq, kv_fmt, k_cache, v_cache, k_scale, v_scale,
                     n_pages, page_size, status, stream);
}

size_t lora_qk_norm_rope_backward_workspace_bytes(int32_t T, int32_t D) { return rope_backward_workspace(T, D); }

lora_status lora_qk_norm_rope_backward(const uint16_t* qkv, int64_t ld, const int32_t* positions, const uint16_t* dq,
                                       const uint16_t* dk, const uint16_t* dv, int32_t T, int32_t n_q, int32_t n_kv,
                                       int32_t D, const float* cos_sin, int32_t max_pos, int32_t rot,
                                       int32_t interleaved, const float* q_weight, const float* k_weight, float eps,
                                       uint16_t* dqkv, int64_t ldd, float* dq_weight, float* dk_weight,
                                       int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  return norm_rope_backward(qkv, ld, positions, {0, nullptr}, dq, dk, dv, T, n_q, n_kv, D, cos_sin, max_pos, rot,
                            interleaved, q_weight, k_weight, eps, dqkv, ldd, dq_weight, dk_weight, status, workspace,
                            workspace_bytes, stream);
}

lora_status lora_qk_norm_rope_axes_backward(const uint16_t* qkv, int64_t ld, const int32_t* positions, int32_t n_axes,
                                            const uint8_t* pair_axes, const uint16_t* dq, const uint16_t* dk,
                                            const uint16_t* dv, int32_t T, int32_t n_q, int32_t n_kv, int32_t D,
                                            const float* cos_sin, int32_t max_pos, int32_t rot, int32_t interleaved,
                                            const float* q_weight, const float* k_weight, float eps, uint16_t* dqkv,
                                            int64_t ldd, float* dq_weight, float* dk_weight, int32_t* status,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  const lora_status st = check_axes(n_axes);
  if (st != LORA_OK) return st;
  return norm_rope_backward(qkv, ld, positions, {n_axes, pair_axes}, dq, dk, dv, T, n_q, n_kv, D, cos_sin, max_pos,
                            rot, interleaved, q_weight, k_weight, eps, dqkv, ldd, dq_weight, dk_weight, status,
                            workspace, workspace_bytes, stream);
}

lora_status lora_tree_mask(const int32_t* parents, const int32_t* q_indptr, int32_t B, int32_t T, int32_t max_q,
                           int32_t words, uint64_t* mask, int32_t* status, void* stream) {
  if (B < 0 || T < 0 || max_q < 0 || words < 1) return LORA_ERR_INVALID_ARG;
  if (B > ATTN_MAX_B || T > MAX_TOKENS || words > MAX_DRAFT_WORDS || max_q > 64 * words) return LORA_ERR_UNSUPPORTED;
  if (T == 0) return LORA_OK;
  if (B == 0 || !parents || !q_indptr || !mask || !aligned(parents, 4) || !aligned(q_indptr, 4) || !aligned(mask, 8) ||
      !aligned(status, 4))
    return LORA_ERR_INVALID_ARG;
  return launch_tree_mask(parents, q_indptr, B, T, max_q, words, mask, status, as_stream(stream)) == hipSuccess
             ? LORA_OK : LORA_ERR_HIP;
}

size_t lora_tree_attention_workspace_bytes(int32_t n_q, int32_t n_kv, int32_t D, int32_t max_q) {
  if (check_heads(1, n_q, n_kv, D) != LORA_OK || n_q % n_kv != 0 || max_q < 1 || max_q > MAX_TOKENS) return 0;
  size_t most = 0;  // of the two cache formats, few sequences and many
  for (int way = 0; way < 4; ++way) {
    const size_t n = plan_bytes(tree_attn_plan(D, max_q, n_q / n_kv, way & 1, false, way & 2 ? (long)ATTN_MAX_B * n_kv : 1));
    most = n > most ? n : most;
  }
  return most;
}

lora_status lora_tree_attention(const uint16_t* q, int64_t ldq, int32_t kv_fmt, const void* k_cache,
                                const void* v_cache, const float* k_scale, const float* v_scale, int32_t n_pages,
                                int32_t page_size, const int32_t* page_table, int32_t max_pages, const int32_t* kv_len,
                                const int32_t* q_indptr, int32_t B, int32_t T, int32_t max_q, int32_t n_q, int32_t n_kv,
                                int32_t D, const uint64_t* tree_mask, int32_t mask_words, float scale, uint16_t* out,
                                float* lse, int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  lora_status st = check_heads(T, n_q, n_kv, D);
  if (st != LORA_OK) return st;
  int32_t lg = 0;
  if (!cache_fmt_ok(kv_fmt) || B < 0 || max_q < 0 || max_pages < 0 || n_q % n_kv != 0 || !isfinite(scale))
    return LORA_ERR_INVALID_ARG;
  if ((st = check_pages(n_pages, page_size, n_kv, &lg)) != LORA_OK) return st;
  if (B > ATTN_MAX_B || max_q > MAX_TOKENS || (int64_t)max_pages * page_size > (1 << 30)) return LORA_ERR_UNSUPPORTED;
  if (tree_mask) {
    if (mask_words < 1) return LORA_ERR_INVALID_ARG;
    if (mask_words > MAX_DRAFT_WORDS || max_q > 64 * mask_words) return LORA_ERR_UNSUPPORTED;
  }
  if (T == 0 || B == 0 || max_q == 0) return LORA_OK;
  if (!rows_ok(q, ldq, (int64_t)n_q * D) || !k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !kv_len || !aligned(kv_len, 4) || !q_indptr || !aligned(q_indptr, 4) || !out || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(tree_mask, 8) || !aligned(status, 4) || max_pages < 1 || !page_table ||
      !aligned(page_table, 4))
    return LORA_ERR_INVALID_ARG;
  const bool fp8 = kv_fmt == LORA_KV_FP8_E4M3;
  if (fp8 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4))) return LORA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)max_q * (n_q / n_kv);
  if (rows > INT32_MAX / 2) return LORA_ERR_UNSUPPORTED;
  const TreeAttnPlan pl = tree_attn_plan(D, max_q, n_q / n_kv, fp8, tree_mask != nullptr, (long)B * n_kv);
  // All steps of a call, which count 3 at most, are numbered in 32 bits.  Its row blocks are every
  // sequence's at max_q rows, or what all T rows fill and a part one for each sequence that has any.
  const double blocks = std::min((double)B * (double)((rows + pl.block_rows - 1) / pl.block_rows),
                                 (double)T * (n_q / n_kv) / pl.block_rows + std::min(B, T));
  const double steps = blocks * n_kv * ((double)max_pages * page_size / ATTN_KEYS + 1.0);
  if (steps > 5.0e8) return LORA_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < lora_tree_attention_workspace_bytes(n_q, n_kv, D, max_q))
    return LORA_ERR_WORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  TreeAttnParams p{};
  p.q = q; p.ldq = ldq; p.k_cache = k_cache; p.v_cache = v_cache;
  p.k_scale = fp8 ? k_scale : nullptr; p.v_scale = fp8 ? v_scale : nullptr;
  p.page_table = page_table; p.max_pages = max_pages; p.n_pages = n_pages; p.page_log2 = lg;
  p.kv_len = kv_len; p.q_indptr = q_indptr; p.B = B; p.T = T; p.max_q = max_q; p.n_q = n_q; p.n_kv = n_kv;
  p.group = n_q / n_kv; p.mask = tree_mask; p.words = tree_mask ? mask_words : 0;
  p.scale_log2 = scale * 1.44269504088896341f;
  p.out = out; p.lse = lse; p.status = status; p.n_wg = pl.n_wg; p.counted = pl.counted;
  p.desc = reinterpret_cast<int*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + round256(pl.desc_bytes));
  p.part_o = reinterpret_cast<float*>(ws + round256(pl.desc_bytes) + round256(pl.ml_bytes));
  return launch_tree_attention(p, pl, D, fp8, as_stream(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // extern "C"
