// One AdamW step over many tensors: the adapters of many tenants, and plain vectors.
//
// Mathematics, for a value p with gradient g, at step t of its group (a tenant):
//   g' = g min(1, largest / (|g over the group| + 1e-6))        (with norms)
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = (1 - rate decay) p - rate / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
// Every product and sum is rounded on its own, in the order above (no fused multiply-add), so that
// a step has one result whatever the compiler joins: an 8-bit state next to a border of its code
// would otherwise depend on it.  Group coefficients are taken in 64 bits and rounded once.
//
// States in 8 bits: blocks of 64 values share a scale (the largest magnitude / 448); a value is an
// e4m3 code.  Of v its root is held, which halves the exponents that a code has to span; a root that
// is not 0 keeps a code that is not (0 would make the next step as large as m / eps).
#include <algorithm>

#include "step_kernels.hpp"
#include "../csrc/device_common.hpp"

#pragma clang fp contract(off)

namespace lora {
namespace {

enum { KIND_PLAIN = LORA_ADAMW_PLAIN, KIND_A = LORA_ADAMW_A, KIND_B = LORA_ADAMW_B };
enum { C_B1, C_NB1, C_B2, C_NB2, C_EPS, C_ROOT, C_KEEP, C_RATE, C_CLIP, C_ON };

constexpr float E4M3_MAX = 448.f;
constexpr float NO_SCALE = 0x1p-100f;  // blocks below it are held as zero: their scale's inverse would overflow

// Values of a tile in LDS, its rows of an odd length: of A, span rows of r | 1, at most for r = 2
// (2,048 rows of 3); of B, r rows of span + 1.
constexpr int ADAMW_LDS = 6144;

// A tile's place: `n4` quads of values, quad i at value `at(i)` of the tensor.
struct Place {
  long base;
  int n4, len4;   // quads in all, and in a row of the tile
  long ld;        // values from one row of the tile to the next
  int n;          // values in all (plain: the last quad may be part filled)
  __device__ __forceinline__ long at(int i, int& row) const {
    row = i / len4;
    return base + row * ld + 4l * (i - row * len4);
  }
};

__device__ __forceinline__ Place place(const lora_adamw_tensor& t, int first) {
  Place p;
  if (t.kind == KIND_A) {          // rows first .. of [K][r], which lie together
    const int rows = min(adamw_tile_span(t.cols), t.rows - first);
    p.n = rows * t.cols;
    p.base = (long)first * t.cols;
    p.n4 = p.len4 = p.n / 4;
    p.ld = 0;
  } else if (t.kind == KIND_B) {   // columns first .. of [r][N]
    const int cols = min(adamw_tile_span(t.rows), t.cols - first);
    p.n = cols * t.rows;
    p.base = first;
    p.n4 = p.n / 4;
    p.len4 = cols / 4;
    p.ld = t.cols;
  } else {
    p.n = min((long)ADAMW_TILE, (long)t.rows * t.cols - first);
    p.base = first;
    p.n4 = p.len4 = (p.n + 3) / 4;
    p.ld = 0;
  }
  return p;
}

__device__ __forceinline__ float4 ld4(const float* p, int n) {  // the first n of 4 values
  if (n >= 4) return *reinterpret_cast<const float4*>(p);
  return make_float4(p[0], n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, 0.f);
}
__device__ __forceinline__ void st4(float* p, const float4& v, int n) {
  if (n >= 4) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    p[0] = v.x;
    if (n > 1) p[1] = v.y;
    if (n > 2) p[2] = v.z;
  }
}
__device__ __forceinline__ uint32_t ld4(const uint8_t* p, int n) {
  if (n >= 4) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t v = p[0];
  if (n > 1) v |= (uint32_t)p[1] << 8;
  if (n > 2) v |= (uint32_t)p[2] << 16;
  return v;
}
__device__ __forceinline__ void st4(uint8_t* p, uint32_t v, int n) {
  if (n >= 4) {
    *reinterpret_cast<uint32_t*>(p) = v;
  } else {
    for (int i = 0; i < n; ++i) p[i] = (uint8_t)(v >> (8 * i));
  }
}

// Sums of the squares of a tile's gradients.
__global__ __launch_bounds__(256) void k_adamw_norms(AdamWParams p) {
  __shared__ double red[4];
  const lora_adamw_tile tile = p.tiles[blockIdx.x];
  const lora_adamw_tensor t = p.tensors[tile.tensor];
  if (p.active && !p.active[t.group]) return;
  const Place at = place(t, tile.first);
  double s = 0.0;
  for (int i = threadIdx.x; i < at.n4; i += 256) {
    int row;
    const float4 g = ld4(t.grad + at.at(i, row), at.n - 4 * i);
    s += (double)g.x * g.x + (double)g.y * g.y + ((double)g.z * g.z + (double)g.w * g.w);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) p.part[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// A group's coefficients (and its norm, its tiles' sums joined in a fixed order); its step counts.
__global__ __launch_bounds__(256) void k_adamw_groups(AdamWParams p) {
  __shared__ double red[4];
  const int g = blockIdx.x;
  const bool active = !p.active || p.active[g];
  double s = 0.0;
  if (p.norm && active)
    for (int i = p.group_first[g] + threadIdx.x; i < p.group_first[g + 1]; i += 256) s += p.part[i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x) return;
  const double* h = p.hyper + (long)g * ADAMW_HYPER;
  float* c = p.coef + (long)g * ADAMW_COEF;
  bool on = active;
  double clip = 1.0;
  if (p.norm) {
    const double norm = sqrt((red[0] + red[1]) + (red[2] + red[3]));
    p.norm[g] = (float)norm;
    if (h[5] > 0.0) clip = fmin(1.0, h[5] / (norm + 1e-6));
    if (!(norm <= 1.7976931348623157e308)) {
      on = false;
      if (p.status) or_agent(p.status, LORA_ADAMW_NOT_FINITE);
    }
  }
  if (on) {
    const int t = p.steps[g] + 1;
    p.steps[g] = t;
    double p1 = 1.0, p2 = 1.0, q1 = h[1], q2 = h[2];
    for (int e = t; e > 0; e >>= 1) {
      if (e & 1) { p1 *= q1; p2 *= q2; }
      q1 *= q1;
      q2 *= q2;
    }
    c[C_B1] = (float)h[1];
    c[C_NB1] = (float)(1.0 - h[1]);
    c[C_B2] = (float)h[2];
    c[C_NB2] = (float)(1.0 - h[2]);
    c[C_EPS] = (float)h[3];
    c[C_ROOT] = (float)(1.0 / sqrt(1.0 - p2));
    c[C_KEEP] = (float)(1.0 - h[0] * h[4]);
    c[C_RATE] = (float)(h[0] / (1.0 - p1));
    c[C_CLIP] = (float)clip;
  }
  c[C_ON] = on ? 1.f : 0.f;
}

__device__ __forceinline__ float sat448(float x) { return x != x ? x : fminf(fmaxf(x, -E4M3_MAX), E4M3_MAX); }
__device__ __forceinline__ uint32_t codes(const float (&v)[4]) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(sat448(v[0]), sat448(v[1]), r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(sat448(v[2]), sat448(v[3]), r, true);
  return (uint32_t)r;
}
__device__ __forceinline__ void values(uint32_t c, float scale, float (&v)[4]) {
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)c, 0) * scale;
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)c, 1) * scale;
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)c, 2) * scale;
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)c, 3) * scale;
}
// Scale of a block from its 16 lanes' quads, and its inverse.
__device__ __forceinline__ void block_scale(const float (&v)[4], float& scale, float& inv) {
  float a = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) a = fmaxf(a, __shfl_xor(a, d));
  a = a >= NO_SCALE ? a : 0.f;
  scale = a * (1.f / E4M3_MAX);
  inv = a > 0.f ? 1.f / a * E4M3_MAX : 0.f;
}

// Eight bf16 of the tile in LDS from (row, col) on, along its rows or its columns; the first n of
// them, the others zero.
template <bool ALONG>
__device__ __forceinline__ uint4 gather8(const uint16_t* s, int ld, int row, int col, int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = 0;
#pragma unroll
    for (int e = 2 * i; e < 2 * i + 2; ++e)
      if (e < n) v |= (uint32_t)(ALONG ? s[row * ld + col + e] : s[(row + e) * ld + col]) << (16 * (e & 1));
    w[i] = v;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A tile's values in the forms that the layer reads.  The tile in LDS has its ranks along the rows
// (RANKS_ALONG: A, [k][j]) or along the columns (B, [j][n]); `first` is its place along the other
// side, of `full` values, of which it has `span`.
template <bool RANKS_ALONG>
__device__ __forceinline__ void write_packs(const uint16_t* s, int ld, int r, int first, int span, int full, uint16_t* operand,
                                            uint16_t* rows) {
  if (operand) {  // MFMA operand order: rank tiles of 16, steps of 64 along the other side
    const int steps = span / 64, chunks = (r + 15) / 16 * steps * 128;
    for (int q = threadIdx.x; q < chunks; q += 256) {
      const int l = q & 63, h = (q >> 6) & 1, st = (q >> 7) % steps, jt = (q >> 7) / steps;
      const int j = 16 * jt + (l & 15), x = 64 * st + 16 * (l >> 4) + 8 * h;
      const uint4 v = RANKS_ALONG ? gather8<false>(s, ld, x, j, j < r ? 8 : 0) : gather8<true>(s, ld, j, x, j < r ? 8 : 0);
      *reinterpret_cast<uint4*>(operand + ((((long)jt * (full / 64) + first / 64 + st) * 2 + h) * 64 + l) * 8) = v;
    }
  }
  if (rows) {     // rows of ranks, padded to a multiple of 8
    const int r8 = (r + 7) / 8, chunks = span * r8;
    for (int q = threadIdx.x; q < chunks; q += 256) {
      const int x = q / r8, j = 8 * (q - x * r8), n = r - j;
      const uint4 v = RANKS_ALONG ? gather8<true>(s, ld, x, j, n) : gather8<false>(s, ld, j, x, n);
      *reinterpret_cast<uint4*>(rows + ((long)(first + x) * r8 * 8 + j)) = v;
    }
  }
}

template <bool BITS8>
__global__ __launch_bounds__(256) void k_adamw(AdamWParams p) {
  __shared__ uint16_t s[ADAMW_LDS];
  const lora_adamw_tile tile = p.tiles[blockIdx.x];
  const lora_adamw_tensor t = p.tensors[tile.tensor];
  const float* c = p.coef + (long)t.group * ADAMW_COEF;
  if (c[C_ON] == 0.f) return;
  const Place at = place(t, tile.first);
  // the tile in LDS: its rows are the tensor's, of an odd length (columns are read too)
  const int ld = (t.kind == KIND_A ? t.cols : 4 * at.len4) | 1;

#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = threadIdx.x + 256 * k, n = at.n - 4 * i;
    const bool live = i < at.n4;
    int row = 0;
    const long o = live ? at.at(i, row) : 0;
    float4 g4 = make_float4(0.f, 0.f, 0.f, 0.f), p4 = g4, m4 = g4, v4 = g4;
    uint32_t mc = 0, vc = 0;
    float ms = 0.f, vs = 0.f;
    if (live) {
      g4 = ld4(t.grad + o, n);
      p4 = ld4(t.param + o, n);
      if (BITS8) {
        mc = ld4(reinterpret_cast<const uint8_t*>(t.m) + o, n);
        vc = ld4(reinterpret_cast<const uint8_t*>(t.v) + o, n);
        ms = t.m_scale[o / ADAMW_BLOCK];
        vs = t.v_scale[o / ADAMW_BLOCK];
      } else {
        m4 = ld4(reinterpret_cast<const float*>(t.m) + o, n);
        v4 = ld4(reinterpret_cast<const float*>(t.v) + o, n);
      }
    }
    float g[4] = {g4.x, g4.y, g4.z, g4.w}, w[4] = {p4.x, p4.y, p4.z, p4.w};
    float m[4] = {m4.x, m4.y, m4.z, m4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w}, root[4];
    if (BITS8) {
      values(mc, ms, m);
      values(vc, vs, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] * v[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ge = p.norm ? g[e] * c[C_CLIP] : g[e];
      m[e] = m[e] * c[C_B1] + ge * c[C_NB1];
      v[e] = v[e] * c[C_B2] + (ge * ge) * c[C_NB2];
      root[e] = sqrtf(v[e]);
      w[e] = w[e] * c[C_KEEP] - (m[e] / (root[e] * c[C_ROOT] + c[C_EPS])) * c[C_RATE];
    }
    if (BITS8) {
      float si, inv;
      block_scale(m, si, inv);
      float q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = m[e] * inv;
      if (live) {
        st4(reinterpret_cast<uint8_t*>(t.m) + o, codes(q), n);
        if ((threadIdx.x & 15) == 0) t.m_scale[o / ADAMW_BLOCK] = si;
      }
      block_scale(root, si, inv);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[e] = root[e] * inv;
        if (root[e] > 0.f && inv > 0.f) q[e] = fmaxf(q[e], 0x1p-9f);  // the least code that is not 0
      }
      if (live) {
        st4(reinterpret_cast<uint8_t*>(t.v) + o, codes(q), n);
        if ((threadIdx.x & 15) == 0) t.v_scale[o / ADAMW_BLOCK] = si;
      }
    } else if (live) {
      st4(reinterpret_cast<float*>(t.m) + o, make_float4(m[0], m[1], m[2], m[3]), n);
      st4(reinterpret_cast<float*>(t.v) + o, make_float4(v[0], v[1], v[2], v[3]), n);
    }
    if (!live) continue;
    st4(t.param + o, make_float4(w[0], w[1], w[2], w[3]), n);
    if (t.copy || t.kind != KIND_PLAIN) {
      const uint32_t lo = bf16x2_rne(w[0], w[1]), hi = bf16x2_rne(w[2], w[3]);
      if (t.copy) {
        if (n >= 4) {
          *reinterpret_cast<uint2*>(t.copy + o) = make_uint2(lo, hi);
        } else {
          t.copy[o] = (uint16_t)lo;
          if (n > 1) t.copy[o + 1] = (uint16_t)(lo >> 16);
          if (n > 2) t.copy[o + 2] = (uint16_t)hi;
        }
      }
      const uint16_t b[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
      if (t.kind == KIND_A) {
        int k0 = 4 * i / t.cols, j = 4 * i - k0 * t.cols;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[k0 * ld + j] = b[e];
          if (++j == t.cols) { j = 0; ++k0; }
        }
      } else if (t.kind == KIND_B) {
        const int x = row * ld + 4 * (i - row * at.len4);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x + e] = b[e];
      }
    }
  }
  if (t.kind == KIND_PLAIN || (!t.pack && !t.pack_bwd)) return;
  __syncthreads();
  if (t.kind == KIND_A) write_packs<true>(s, ld, t.cols, tile.first, at.n / t.cols, t.rows, t.pack, t.pack_bwd);
  else write_packs<false>(s, ld, t.rows, tile.first, 4 * at.len4, t.cols, t.pack_bwd, t.pack);
}

}  // namespace

hipError_t launch_adamw(const AdamWParams& p, int state_bits, hipStream_t s) {
  if (p.norm && p.n_tiles) hipLaunchKernelGGL(k_adamw_norms, dim3((unsigned)p.n_tiles), dim3(256), 0, s, p);
  hipLaunchKernelGGL(k_adamw_groups, dim3(p.n_groups), dim3(256), 0, s, p);
  if (p.n_tiles) {
    if (state_bits == 8) hipLaunchKernelGGL(k_adamw<true>, dim3((unsigned)p.n_tiles), dim3(256), 0, s, p);
    else hipLaunchKernelGGL(k_adamw<false>, dim3((unsigned)p.n_tiles), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace lora
