// Host layer of the norms and of the AdamW step: argument checks and launches.  Every check runs
// before anything is enqueued; nothing here synchronises, and no call that enqueues allocates.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <exception>
#include <vector>

#include "step_kernels.hpp"

using namespace lora;

namespace {

constexpr int MAX_TOKENS = 65536;
constexpr int MAX_GROUPS = 8192;
constexpr int MAX_TENSORS = 1 << 20;
constexpr int64_t MAX_TILES = (1 << 22) - 1;  // of 1,024 threads: a launch has fewer than 2^32

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// bf16 rows read and written in 16-byte pieces.
inline bool rows_ok(const void* p, int64_t ld, int64_t width) { return p && aligned(p, 16) && ld >= width && ld % 8 == 0; }

lora_status check_norm(int32_t T, int32_t K, float eps, int32_t rms) {
  if (T < 0 || K < 1 || !(eps >= 0.f) || !isfinite(eps) || (rms != 0 && rms != 1)) return LORA_ERR_INVALID_ARG;
  return T > MAX_TOKENS || K > NORM_MAX_K || K % 8 != 0 ? LORA_ERR_UNSUPPORTED : LORA_OK;
}

lora_status check_tensor(const lora_adamw_tensor& t, int32_t n_groups, int32_t bits) {
  if (!t.param || !t.grad || !t.m || !t.v || t.rows < 1 || t.cols < 1 || t.group < 0 || t.group >= n_groups)
    return LORA_ERR_INVALID_ARG;
  const void* wide[] = {t.param, t.grad, t.m, t.v, t.copy, t.pack, t.pack_bwd};
  for (const void* p : wide)
    if (!aligned(p, 16)) return LORA_ERR_INVALID_ARG;
  if (bits == 8 ? !t.m_scale || !t.v_scale || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4) : t.m_scale || t.v_scale)
    return LORA_ERR_INVALID_ARG;
  if ((int64_t)t.rows * t.cols > INT32_MAX - 4096) return LORA_ERR_UNSUPPORTED;
  switch (t.kind) {
    case LORA_ADAMW_PLAIN: return t.pack || t.pack_bwd ? LORA_ERR_INVALID_ARG : LORA_OK;
    case LORA_ADAMW_A: return t.cols > 64 || t.rows % 64 != 0 ? LORA_ERR_UNSUPPORTED : LORA_OK;
    case LORA_ADAMW_B: return t.rows > 64 || t.cols % 64 != 0 ? LORA_ERR_UNSUPPORTED : LORA_OK;
    default: return LORA_ERR_INVALID_ARG;
  }
}

// The side that a tensor is cut along, and the values of it that a tile takes.
void cut(const lora_adamw_tensor& t, int64_t& side, int64_t& span) {
  if (t.kind == LORA_ADAMW_A) {
    side = t.rows;
    span = adamw_tile_span(t.cols);
  } else if (t.kind == LORA_ADAMW_B) {
    side = t.cols;
    span = adamw_tile_span(t.rows);
  } else {
    side = (int64_t)t.rows * t.cols;
    span = ADAMW_TILE;
  }
}

struct Range { uintptr_t first, last; bool written; };

// Whether a range that a step writes overlaps another.
bool overlap(const lora_adamw_tensor* t, int32_t n, int32_t bits) {
  std::vector<Range> all;
  all.reserve((size_t)n * 9);
  auto add = [&](const void* p, size_t bytes, bool written) {
    if (p) all.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, written});
  };
  for (int32_t i = 0; i < n; ++i) {
    const size_t v = (size_t)t[i].rows * t[i].cols;
    add(t[i].param, 4 * v, true);
    add(t[i].grad, 4 * v, false);
    add(t[i].m, bits / 8 * v, true);
    add(t[i].v, bits / 8 * v, true);
    add(t[i].m_scale, (v + 63) / 64 * 4, true);
    add(t[i].v_scale, (v + 63) / 64 * 4, true);
    add(t[i].copy, 2 * v, true);
    const size_t r = t[i].kind == LORA_ADAMW_A ? t[i].cols : t[i].rows, side = t[i].kind == LORA_ADAMW_A ? t[i].rows : t[i].cols;
    const size_t operand = (r + 15) / 16 * 32 * side, rows = (r + 7) / 8 * 16 * side;
    add(t[i].pack, t[i].kind == LORA_ADAMW_A ? operand : rows, true);
    add(t[i].pack_bwd, t[i].kind == LORA_ADAMW_A ? rows : operand, true);
  }
  std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.first < b.first; });
  // the furthest ends so far, of those written and of all
  uintptr_t written = 0, any = 0;
  for (const Range& r : all) {
    if (r.first < written || (r.written && r.first < any)) return true;
    any = std::max(any, r.last);
    if (r.written) written = std::max(written, r.last);
  }
  return false;
}

}  // namespace

extern "C" {

lora_status lora_layer_norm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr, int32_t T, int32_t K,
                            const float* weight, const float* bias, float eps, int32_t rms, uint16_t* y, int64_t ldy,
                            uint16_t* sum, int64_t lds, void* stream) {
  const lora_status st = check_norm(T, K, eps, rms);
  if (st != LORA_OK || T == 0) return st;
  if (!rows_ok(x, ldx, K) || !rows_ok(y, ldy, K) || !aligned(weight, 16) || !aligned(bias, 16) ||
      (residual == nullptr) != (sum == nullptr) || (sum && sum == y) || (residual && (!rows_ok(residual, ldr, K) || !rows_ok(sum, lds, K))))
    return LORA_ERR_INVALID_ARG;
  NormParams p{x, ldx, residual, ldr, T, K, weight, bias, eps, y, ldy, sum, lds};
  return launch_norm(p, rms, as_stream(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

size_t lora_layer_norm_backward_workspace_bytes(int32_t T, int32_t K) {
  if (T < 1 || check_norm(T, K, 0.f, 0) != LORA_OK) return 0;
  return (size_t)std::min(T, NORM_BWD_WGS) * 2 * K * sizeof(float);
}

lora_status lora_layer_norm_backward(const uint16_t* dy, int64_t lddy, const uint16_t* h, int64_t ldh,
                                     const float* weight, const uint16_t* dsum, int64_t ldds, int32_t T, int32_t K,
                                     float eps, int32_t rms, uint16_t* dx, int64_t lddx, float* dweight, float* dbias,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  const lora_status st = check_norm(T, K, eps, rms);
  if (st != LORA_OK) return st;
  if (!aligned(dweight, 16) || !aligned(dbias, 16)) return LORA_ERR_INVALID_ARG;
  if (T > 0) {
    if (!rows_ok(dy, lddy, K) || !rows_ok(h, ldh, K) || !rows_ok(dx, lddx, K) || (dsum && !rows_ok(dsum, ldds, K)) ||
        !aligned(weight, 16))
      return LORA_ERR_INVALID_ARG;
    if ((dweight || dbias) && (!workspace || !aligned(workspace, 16) ||
                               workspace_bytes < lora_layer_norm_backward_workspace_bytes(T, K)))
      return LORA_ERR_WORKSPACE;
  }
  NormBwdParams p{dy, lddy, h, ldh, weight, dsum, ldds, T, K, eps, dx, lddx, dweight, dbias,
                  reinterpret_cast<float*>(workspace), 0};
  return launch_norm_bwd(p, rms, as_stream(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

lora_status lora_adamw_plan(const lora_adamw_tensor* tensors, int32_t n, int32_t n_groups, int32_t state_bits,
                            int64_t* n_tiles, lora_adamw_tile* tiles, int32_t* group_first) {
  if (n < 0 || n_groups < 1 || (n > 0 && !tensors) || !n_tiles || (state_bits != 32 && state_bits != 8) ||
      (tiles && !group_first))
    return LORA_ERR_INVALID_ARG;
  if (n > MAX_TENSORS || n_groups > MAX_GROUPS) return LORA_ERR_UNSUPPORTED;
  try {
    std::vector<int64_t> first((size_t)n_groups + 1, 0);  // tiles of each group, then its next tile's place
    for (int32_t i = 0; i < n; ++i) {
      const lora_status st = check_tensor(tensors[i], n_groups, state_bits);
      if (st != LORA_OK) return st;
      int64_t side, span;
      cut(tensors[i], side, span);
      first[tensors[i].group + 1] += (side + span - 1) / span;
    }
    if (overlap(tensors, n, state_bits)) return LORA_ERR_INVALID_ARG;
    for (int32_t g = 0; g < n_groups; ++g) first[g + 1] += first[g];
    const int64_t all = first[n_groups];
    if (all > MAX_TILES) return LORA_ERR_UNSUPPORTED;
    if (!tiles) {
      *n_tiles = all;
      return LORA_OK;
    }
    if (*n_tiles != all) return LORA_ERR_INVALID_ARG;
    for (int32_t g = 0; g <= n_groups; ++g) group_first[g] = (int32_t)first[g];
    for (int32_t i = 0; i < n; ++i) {
      int64_t side, span;
      cut(tensors[i], side, span);
      for (int64_t at = 0; at < side; at += span) tiles[first[tensors[i].group]++] = {tensors[i], (int32_t)at, 0};
    }
    return LORA_OK;
  } catch (const std::exception&) {  // no host memory for it
    return LORA_ERR_WORKSPACE;
  }
}

size_t lora_adamw_workspace_bytes(int64_t n_tiles, int32_t n_groups) {
  if (n_tiles < 0 || n_tiles > MAX_TILES || n_groups < 1 || n_groups > MAX_GROUPS) return 0;
  return round256((size_t)n_tiles * sizeof(double)) + round256((size_t)n_groups * ADAMW_COEF * sizeof(float)) +
         (size_t)n_groups * ADAMW_LINE * sizeof(int);
}

lora_status lora_adamw_step(const lora_adamw_tile* tiles, int64_t n_tiles, const int32_t* group_first, int32_t n_groups,
                            int32_t state_bits, const double* hyper, const int32_t* active, int32_t* steps,
                            float* grad_norm, int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  if (n_tiles < 0 || n_groups < 1 || (state_bits != 32 && state_bits != 8)) return LORA_ERR_INVALID_ARG;
  if (n_tiles > MAX_TILES || n_groups > MAX_GROUPS) return LORA_ERR_UNSUPPORTED;
  if ((n_tiles > 0 && !tiles) || !aligned(tiles, 8) || !group_first ||
      !aligned(group_first, 4) || !hyper || !aligned(hyper, 8) || !aligned(active, 4) || !steps || !aligned(steps, 4) ||
      !aligned(grad_norm, 4) || !aligned(status, 4))
    return LORA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < lora_adamw_workspace_bytes(n_tiles, n_groups))
    return LORA_ERR_WORKSPACE;
  AdamWParams p{};
  p.tiles = tiles; p.n_tiles = n_tiles; p.group_first = group_first; p.n_groups = n_groups;
  p.hyper = hyper; p.active = active; p.steps = steps; p.norm = grad_norm; p.status = status;
  p.part = reinterpret_cast<double*>(workspace);
  p.coef = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + round256((size_t)n_tiles * sizeof(double)));
  p.arrived = reinterpret_cast<int*>(reinterpret_cast<char*>(p.coef) + round256((size_t)n_groups * ADAMW_COEF * sizeof(float)));
  return launch_adamw(p, state_bits, as_stream(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // extern "C"
