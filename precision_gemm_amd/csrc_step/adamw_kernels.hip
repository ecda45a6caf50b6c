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
// States in 8 bits: blocks of 64 values share a scale (the largest finite magnitude / 448); a value is an
// e4m3 code, NaN's for what is not finite.  Of v its root is held, which halves the exponents that a code
// has to span; a root that is not 0 keeps a code that is not (0 would make the next step as large as m / eps).
//
// Bound by HBM: 59 instructions a value with states in 32 bits, 95 in 8, beside 28 and 16 bytes of
// states and master copies and 6 of bf16 forms.  A workgroup takes a tile whose bf16 form it has in LDS,
// so that the packed forms, one of which is always across the tensor's rows, leave in whole 16-byte
// pieces in the same pass (repacking by launches of their own would be two for each adapter).  32 tenants of rank 16
// on four projections (35.7 million values, 1.21 GB; 0.79 in 8 bits): 195 us, 6.2 TB/s, and 147, 5.4; a
// copy of as many bytes reaches 5.1.
#include <algorithm>

#include "step_kernels.hpp"
#include "../csrc/device_common.hpp"

#pragma clang fp contract(off)

namespace lora {
namespace {

enum { KIND_PLAIN = LORA_ADAMW_PLAIN, KIND_A = LORA_ADAMW_A, KIND_B = LORA_ADAMW_B };
// Values of a tile in LDS: of A, span rows of r + 4; of B, r rows of span + 8.
constexpr int ADAMW_LDS = 5120;

constexpr float E4M3_MAX = 448.f, F32_MAX = 3.402823466e38f;
constexpr float NO_SCALE = 0x1p-100f;  // blocks below it are held as zero: their scale's inverse would overflow

// A tile's place: `n4` quads of values, quad i at value at(i) of the tensor.
struct Place {
  long base;
  int n;          // values in all (plain: the last quad may be part filled)
  int n4, len4;   // quads in all, and in a row of the tile
  unsigned inv;   // 2^20 / len4, rounded up: i / len4 = i inv >> 20 for i < 1024
  long ld;        // values from one row of the tile to the next
  __device__ __forceinline__ int row(int i) const { return (int)((unsigned)i * inv >> 20); }
  __device__ __forceinline__ long at(int i) const {
    const int r = row(i);
    return base + r * ld + 4 * (i - r * len4);
  }
};

__device__ __forceinline__ Place place(const lora_adamw_tensor& t, int first) {
  Place p;
  if (t.kind == KIND_B) {   // columns first .. of [r][N]
    const int cols = min(adamw_tile_span(t.rows), t.cols - first);
    p.n = cols * t.rows;
    p.base = first;
    p.len4 = cols / 4;
    p.inv = (1u << 20) / (unsigned)p.len4 + 1;
    p.ld = t.cols;
  } else {                  // values that lie together: rows first .. of [K][r], or values of a vector
    const bool a = t.kind == KIND_A;
    p.n = a ? min(adamw_tile_span(t.cols), t.rows - first) * t.cols : (int)min((long)ADAMW_TILE, (long)t.rows * t.cols - first);
    p.base = a ? (long)first * t.cols : first;
    p.len4 = 0;
    p.inv = 0;
    p.ld = 0;
  }
  p.n4 = (p.n + 3) / 4;
  return p;
}

// Addresses come out of memory: stated to be global ones, so that their loads and stores are (a flat
// access also counts as one of LDS, whose waits would wait for it).
// PAST: past the caches (see STREAM_TILES).
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <typename T, bool PAST = false>
__device__ __forceinline__ T ldg(const void* p) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(1))) const T g_t;
  g_t* at = (g_t*)(reinterpret_cast<uintptr_t>(p));
  if constexpr (PAST) return __builtin_nontemporal_load(at);
  else return *at;
#else
  return *reinterpret_cast<const T*>(p);  // host pass only; never executed
#endif
}
template <bool PAST = false, typename T>
__device__ __forceinline__ void stg(void* p, const T& v) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(1))) T g_t;
  g_t* at = (g_t*)(reinterpret_cast<uintptr_t>(p));
  if constexpr (PAST) __builtin_nontemporal_store(v, at);
  else *at = v;
#else
  *reinterpret_cast<T*>(p) = v;
#endif
}

__device__ __forceinline__ float4 as_float4(const f32x4& v) { return make_float4(v.x, v.y, v.z, v.w); }

// Four values at p, or with PART the first n of them (a vector's last).
template <bool PART, bool PAST>
__device__ __forceinline__ float4 ld4(const float* p, int n) {
  if (!PART || n >= 4) return as_float4(ldg<f32x4, PAST>(p));
  return make_float4(n > 0 ? ldg<float>(p) : 0.f, n > 1 ? ldg<float>(p + 1) : 0.f, n > 2 ? ldg<float>(p + 2) : 0.f, 0.f);
}
template <bool PART, bool PAST>
__device__ __forceinline__ uint32_t ld4(const uint8_t* p, int n) {
  if (!PART || n >= 4) return ldg<uint32_t, PAST>(p);
  uint32_t v = 0;
  for (int i = 0; i < n; ++i) v |= (uint32_t)ldg<uint8_t>(p + i) << (8 * i);
  return v;
}
template <bool PART, bool PAST>
__device__ __forceinline__ void st4(float* p, const float (&v)[4], int n) {
  if (!PART || n >= 4) return stg<PAST>(p, f32x4{v[0], v[1], v[2], v[3]});
  if (n > 0) stg(p, v[0]);
  if (n > 1) stg(p + 1, v[1]);
  if (n > 2) stg(p + 2, v[2]);
}
template <bool PART, bool PAST>
__device__ __forceinline__ void st4(uint8_t* p, uint32_t v, int n) {
  if (!PART || n >= 4) return stg<PAST>(p, v);
  for (int i = 0; i < n; ++i) stg(p + i, (uint8_t)(v >> (8 * i)));
}
template <bool PART>
__device__ __forceinline__ void st4(uint16_t* p, const uint2& v, int n) {
  if (!PART || n >= 4) return stg(p, v);
  if (n > 0) stg(p, (uint16_t)v.x);
  if (n > 1) stg(p + 1, (uint16_t)(v.x >> 16));
  if (n > 2) stg(p + 2, (uint16_t)v.y);
}

// A group's coefficients at step t.
struct Coef { float b1, nb1, b2, nb2, eps, root, keep, rate, clip; };

__device__ __forceinline__ Coef coefficients(const double* h, int t, double clip) {
  double p1 = 1.0, p2 = 1.0, q1 = h[1], q2 = h[2];  // beta1^t and beta2^t by squaring
  for (int e = t; e > 0; e >>= 1) {
    if (e & 1) { p1 *= q1; p2 *= q2; }
    q1 *= q1;
    q2 *= q2;
  }
  Coef c;
  c.b1 = (float)h[1];
  c.nb1 = (float)(1.0 - h[1]);
  c.b2 = (float)h[2];
  c.nb2 = (float)(1.0 - h[2]);
  c.eps = (float)h[3];
  c.root = (float)(1.0 / sqrt(1.0 - p2));
  c.keep = (float)(1.0 - h[0] * h[4]);
  c.rate = (float)(h[0] / (1.0 - p1));
  c.clip = (float)clip;
  return c;
}
__device__ __forceinline__ void put(float* to, const Coef& c, bool on) {
  to[0] = c.b1; to[1] = c.nb1; to[2] = c.b2; to[3] = c.nb2; to[4] = c.eps; to[5] = c.root; to[6] = c.keep; to[7] = c.rate;
  to[8] = c.clip; to[9] = on ? 1.f : 0.f;
}
// The same through the scalar cache (an earlier launch wrote them).
typedef __attribute__((address_space(4))) const float c_float;
__device__ __forceinline__ Coef get(const float* c) { return {c[0], c[1], c[2], c[3], c[4], c[5], c[6], c[7], c[8]}; }
__device__ __forceinline__ Coef get(c_float* c) { return {c[0], c[1], c[2], c[3], c[4], c[5], c[6], c[7], c[8]}; }

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  return s;
}

// Settles a group from the sum of its gradients' squares: norm, step, coefficients.  One thread.
__device__ __forceinline__ void settle(const AdamWParams& p, int g, bool on, double sum) {
  const double* h = p.hyper + (long)g * ADAMW_HYPER;
  double clip = 1.0;
  if (p.norm) {
    const double norm = sqrt(sum);
    p.norm[g] = (float)norm;
    if (h[5] > 0.0) clip = fmin(1.0, h[5] / (norm + 1e-6));
    if (!(norm <= 1.7976931348623157e308)) {
      on = false;
      if (p.status) or_agent(p.status, LORA_ADAMW_NOT_FINITE);
    }
  }
  const int step = p.steps[g] + 1;
  if (on) p.steps[g] = step;
  put(p.coef + (long)g * ADAMW_COEF, coefficients(h, step, clip), on);
}

// Sums of the squares of the tiles' gradients, a wave a tile, all its loads in flight at once.  35.7
// million gradients (143 MB) behind an update: 38 us, 3.8 TB/s, with that update's stores still on
// their way to memory (alone 31 us, 4.6); two or four waves a tile do not change it.
// LAST: the wave that is the last of its group settles the group (its sums in their order, whichever
// wave that is), and workgroups behind the tiles' settle the groups that make no step.
template <bool LAST>
__global__ __launch_bounds__(256) void k_adamw_norms(AdamWParams p) {
  const int lane = threadIdx.x & 63;
  const long n_wg = (p.n_tiles + 3) / 4;
  if (LAST && blockIdx.x >= n_wg) {
    const int g = (int)(blockIdx.x - n_wg) * 256 + threadIdx.x;
    if (g < p.n_groups && ((p.active && !p.active[g]) || p.group_first[g] == p.group_first[g + 1])) settle(p, g, false, 0.0);
    return;
  }
  const long at = (long)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (at >= p.n_tiles) return;
  const lora_adamw_tile tile = p.tiles[at];
  const lora_adamw_tensor& t = tile.tensor;
  if (p.active && !p.active[t.group]) return;
  const Place pl = place(t, tile.first);
  const int full = pl.n >> 2;
  f32x4 g[16];
  // lanes without a quad read the tile's first: a load under a condition would wait for the one before
  if (full) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int i = lane + 64 * k;
      g[k] = ldg<f32x4>(t.grad + pl.at(i < full ? i : 0));
    }
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const double q = ((double)g[k].x * g[k].x + (double)g[k].y * g[k].y) + ((double)g[k].z * g[k].z + (double)g[k].w * g[k].w);
    s += lane + 64 * k < full ? q : 0.0;
  }
  if ((pl.n & 3) && lane == 0) {
    const float4 e = ld4<true, false>(t.grad + pl.at(full), pl.n & 3);
    s += (double)e.x * e.x + (double)e.y * e.y + (double)e.z * e.z;
  }
  s = wave_sum(s);
  if (!LAST) {
    if (lane == 0) p.part[at] = s;
    return;
  }
  const int first = p.group_first[t.group], last = p.group_first[t.group + 1];
  int before = 0;
  if (lane == 0) {
    st_agent_u64(reinterpret_cast<uint64_t*>(p.part + at), __builtin_bit_cast(uint64_t, s));
    wait_stores();
    before = add_agent(p.arrived + ADAMW_LINE * t.group, 1);
  }
  if (__builtin_amdgcn_readfirstlane(before) != last - first - 1) return;
  s = 0.0;
  for (int i = first + lane; i < last; i += 64)
    s += __builtin_bit_cast(double, ld_agent_u64(reinterpret_cast<const uint64_t*>(p.part + i)));
  s = wave_sum(s);
  if (lane) return;
  set_agent(p.arrived + ADAMW_LINE * t.group, 0);
  settle(p, t.group, true, s);
}

// The groups, a workgroup each, where the norms' launch does not settle them (or there is none).
__global__ __launch_bounds__(256) void k_adamw_groups(AdamWParams p) {
  __shared__ double red[4];
  const int g = blockIdx.x, first = p.group_first[g], last = p.group_first[g + 1];
  const bool on = (!p.active || p.active[g]) && first != last;
  double s = 0.0;
  if (p.norm && on) {
#pragma unroll 8
    for (int i = first + threadIdx.x; i < last; i += 256) s += p.part[i];
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) settle(p, g, on, (red[0] + red[1]) + (red[2] + red[3]));
}

// e4m3 codes, to nearest even.  No clamp: a value is at most its block's largest times 448 / largest, a
// rounding or two above 448, which the conversion takes to 448 (what would round past it begins at 464).
__device__ __forceinline__ uint32_t codes(const float (&v)[4]) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true);
  return (uint32_t)r;
}
__device__ __forceinline__ void values(uint32_t c, float scale, float (&v)[4]) {
  v[0] = __builtin_amdgcn_cvt_f32_fp8((int)c, 0) * scale;
  v[1] = __builtin_amdgcn_cvt_f32_fp8((int)c, 1) * scale;
  v[2] = __builtin_amdgcn_cvt_f32_fp8((int)c, 2) * scale;
  v[3] = __builtin_amdgcn_cvt_f32_fp8((int)c, 3) * scale;
}
// Largest magnitude of a block from its 16 lanes' quads (a row of lanes); NaN counts for nothing.
template <int CTRL>
__device__ __forceinline__ float row_max(float a) {
  return fmaxf(a, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, a), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ float block_max(const float (&v)[4]) {
  float a = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
  a = row_max<0xb1>(a);          // its neighbour
  a = row_max<0x4e>(a);          // the other pair of four
  a = row_max<0x141>(a);         // the other four of eight
  return row_max<0x140>(a);      // the other eight
}
// Scale of a block, and its inverse.
__device__ __forceinline__ void block_scale(const float (&v)[4], float& scale, float& inv) {
  float a = block_max(v);
  a = a >= NO_SCALE ? a : 0.f;  // (of nothing but NaN: NaN, so 0)
  scale = a * (1.f / E4M3_MAX);
  inv = a > 0.f ? 1.f / a * E4M3_MAX : 0.f;
}

// A quad of its block's moments and roots as it is held in 8 bits.
struct Held { float ms, vs; uint32_t m, v; };
__device__ __forceinline__ Held hold(const float (&m)[4], const float (&root)[4]) {
  Held h;
  float inv, q[4];
  block_scale(m, h.ms, inv);
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = m[e] * inv;
  h.m = codes(q);
  block_scale(root, h.vs, inv);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    q[e] = root[e] * inv;
    if (root[e] > 0.f && inv > 0.f) q[e] = fmaxf(q[e], 0x1p-9f);  // the least code that is not 0
  }
  h.v = codes(q);
  return h;
}
// What is infinite (of an infinite gradient, or of one whose square is) becomes NaN, which counts for
// nothing in its block.
__device__ __forceinline__ void no_infinity(float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (!(fabsf(v[e]) <= F32_MAX)) v[e] = __builtin_nanf("");
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

// The tile of A ([k][j], rows first .. of K) in At's order, from LDS; and in rows of ranks padded to a
// multiple of 8, where those are not the tile as it is.
template <int WG>
__device__ __forceinline__ void write_packs_a(const uint16_t* s, int ld, int r, int first, int span, int K, uint16_t* operand,
                                              uint16_t* rows) {
  const int l = threadIdx.x & 63, h = (threadIdx.x >> 6) & 1, steps = span / 64;
  if (operand) {  // rank tiles of 16, steps of 64 along K, 128 chunks of eight k each
    const int x0 = 16 * (l >> 4) + 8 * h, all = (r + 15) / 16 * steps;
    for (int q = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 7); q < all; q += WG / 128) {
      const int jt = q / steps, st = q - jt * steps, j = 16 * jt + (l & 15);
      const uint4 v = gather8<false>(s, ld, 64 * st + x0, j, j < r ? 8 : 0);
      stg(operand + ((((long)jt * (K / 64) + first / 64 + st) * 2 + h) * 64 + l) * 8, v);
    }
  }
  if (rows) {
    const int r8 = (r + 7) / 8, inv = (1 << 16) / r8 + 1;  // q / r8 = q inv >> 16 for q < 2048
    for (int q = threadIdx.x; q < span * r8; q += WG) {
      const int x = q * inv >> 16, j = 8 * (q - x * r8);
      stg(rows + ((long)(first + x) * r8 * 8 + j), gather8<true>(s, ld, x, j, r - j));
    }
  }
}

// The tile of B ([j][n], columns first .. of N) in Bop's order, and as B^T in rows of ranks.
template <int WG>
__device__ __forceinline__ void write_packs_b(const uint16_t* s, int ld, int r, int first, int span, int N, uint16_t* operand,
                                              uint16_t* rows) {
  const int l = threadIdx.x & 63, h = (threadIdx.x >> 6) & 1, steps = span / 64;
  if (operand) {
    const int x0 = 16 * (l >> 4) + 8 * h, all = (r + 15) / 16 * steps;
    for (int q = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 7); q < all; q += WG / 128) {
      const int jt = q / steps, st = q - jt * steps, j = 16 * jt + (l & 15);
      uint4 v = zero4();
      if (j < r) v = *reinterpret_cast<const uint4*>(s + j * ld + 64 * st + x0);
      stg(operand + ((((long)jt * (N / 64) + first / 64 + st) * 2 + h) * 64 + l) * 8, v);
    }
  }
  if (rows) {
    const int r8 = (r + 7) / 8, inv = (1 << 16) / r8 + 1;
    for (int q = threadIdx.x; q < span * r8; q += WG) {
      const int x = q * inv >> 16, j = 8 * (q - x * r8);
      stg(rows + ((long)(first + x) * r8 * 8 + j), gather8<false>(s, ld, j, x, r - j));
    }
  }
}

// The update of a tile in the registers of WG threads, and its bf16 form into LDS.  PART: the tile is the
// end of a vector of no whole number of blocks; lanes behind the end are nothing to the last block's scale.
template <bool BITS8, bool CLIP, bool PAST, int WG, bool PART, typename GetCoef>
__device__ __forceinline__ void update(const lora_adamw_tensor& t, const Place& at, uint16_t* s, int ld, bool pack_a, bool pack_b,
                                       GetCoef&& get_coef) {
  constexpr int Q = ADAMW_TILE / 4 / WG;
  float4 g4[Q], p4[Q], m4[Q], v4[Q];
  uint32_t mc[Q], vc[Q];
  float ms[Q], vs[Q];
  // Waves without a quad only take part in the barriers.  In the others all loads come first; a lane
  // without a quad reads the tile's first, since a load under a condition would wait for those before it.
  const bool idle = __builtin_amdgcn_readfirstlane((int)threadIdx.x & ~63) >= at.n4;
#pragma unroll
  for (int k = 0; k < Q; ++k) {
    if (idle) break;
    const int i = threadIdx.x + WG * k, n = i < at.n4 ? at.n - 4 * i : PART ? 0 : 4;
    const long o = at.at(i < at.n4 ? i : 0);
    if (BITS8) {
      mc[k] = ld4<PART, false>(reinterpret_cast<const uint8_t*>(t.m) + o, n);
      vc[k] = ld4<PART, false>(reinterpret_cast<const uint8_t*>(t.v) + o, n);
      ms[k] = ldg<float>(t.m_scale + o / ADAMW_BLOCK);
      vs[k] = ldg<float>(t.v_scale + o / ADAMW_BLOCK);
    } else {
      m4[k] = ld4<PART, PAST>(reinterpret_cast<const float*>(t.m) + o, n);
      v4[k] = ld4<PART, PAST>(reinterpret_cast<const float*>(t.v) + o, n);
    }
    g4[k] = ld4<PART, false>(t.grad + o, n);
    p4[k] = ld4<PART, PAST>(t.param + o, n);
  }
  const Coef c = get_coef();
  if (idle) return;
  const bool quads = t.cols % 4 == 0;
  const unsigned by_rank = (1u << 20) / (unsigned)max(1, min(t.cols, 64)) + 1;  // i / r of A, for i < 4096

#pragma unroll
  for (int k = 0; k < Q; ++k) {
    const int i = threadIdx.x + WG * k, n = at.n - 4 * i;
    if (Q > 1 && 4 * WG * k >= at.n) break;
    const bool live = i < at.n4;
    const long o = at.at(i);
    const float g[4] = {g4[k].x, g4[k].y, g4[k].z, g4[k].w};
    float w[4] = {p4[k].x, p4[k].y, p4[k].z, p4[k].w};
    float m[4], v[4], root[4];
    if (BITS8) {
      values(mc[k], ms[k], m);
      values(vc[k], vs[k], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] * v[e];
    } else {
      m[0] = m4[k].x; m[1] = m4[k].y; m[2] = m4[k].z; m[3] = m4[k].w;
      v[0] = v4[k].x; v[1] = v4[k].y; v[2] = v4[k].z; v[3] = v4[k].w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ge = CLIP ? g[e] * c.clip : g[e];
      m[e] = m[e] * c.b1 + ge * c.nb1;
      v[e] = v[e] * c.b2 + (ge * ge) * c.nb2;
      root[e] = sqrtf(v[e]);
      w[e] = w[e] * c.keep - (m[e] / (root[e] * c.root + c.eps)) * c.rate;
    }
    if (BITS8) {
      if (PART) {  // a vector's end: what lies behind it is nothing to its block
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e >= n) m[e] = root[e] = 0.f;
      }
      Held h = hold(m, root);
      // An infinite scale would make the whole block 0 * infinity at the next step.  Asked of the wave, so
      // that a block's lanes stay together, and of the result, so that the scales need not wait for it (32
      // tenants 179 us with it and without, odd ranks 18.4 and 18.0; asked before the codes 180 and 18.7).
      if (__builtin_expect(__any(fmaxf(h.ms, h.vs) > F32_MAX), 0)) {
        no_infinity(m);
        no_infinity(root);
        h = hold(m, root);
      }
      if (!live) continue;
      st4<PART, false>(reinterpret_cast<uint8_t*>(t.m) + o, h.m, n);
      st4<PART, false>(reinterpret_cast<uint8_t*>(t.v) + o, h.v, n);
      if ((threadIdx.x & 15) == 0) {
        stg(t.m_scale + o / ADAMW_BLOCK, h.ms);
        stg(t.v_scale + o / ADAMW_BLOCK, h.vs);
      }
    } else {
      if (!live) continue;
      st4<PART, PAST>(reinterpret_cast<float*>(t.m) + o, m, n);
      st4<PART, PAST>(reinterpret_cast<float*>(t.v) + o, v, n);
    }
    st4<PART, PAST>(t.param + o, w, n);
    const uint2 b = make_uint2(bf16x2_rne(w[0], w[1]), bf16x2_rne(w[2], w[3]));
    if (t.copy) st4<PART>(t.copy + o, b, n);
    if (PART) continue;
    if (pack_a) {
      if (t.pack_bwd && t.cols % 8 == 0) stg(t.pack_bwd + o, b);  // rows without padding
      int k0 = (int)((unsigned)(4 * i) * by_rank >> 20), j = 4 * i - k0 * t.cols;
      if (quads) {
        *reinterpret_cast<uint2*>(s + k0 * ld + j) = b;
      } else {
        const uint16_t each[4] = {(uint16_t)b.x, (uint16_t)(b.x >> 16), (uint16_t)b.y, (uint16_t)(b.y >> 16)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[k0 * ld + j] = each[e];
          if (++j == t.cols) { j = 0; ++k0; }
        }
      }
    } else if (pack_b) {
      const int row = at.row(i);
      *reinterpret_cast<uint2*>(s + row * ld + 4 * (i - row * at.len4)) = b;
    }
  }
}

// A workgroup a tile, a quad a thread: 1,024 threads (256 with four quads each, and 512 with two, took 3 %
// and 1.5 % longer on the layer above, 6.4 and 5.8 us against 5.4 on one adapter of rank 8: more code to
// fetch for fewer waves).  ALONE: the launch is the whole step (no norms, few tiles): every workgroup works
// out its group's coefficients while its loads are in flight, and the group's last counts its step.
template <bool BITS8, bool CLIP, bool ALONE, bool PAST, int WG>
__global__ __launch_bounds__(WG) void k_adamw(AdamWParams p) {
  __shared__ __attribute__((aligned(16))) uint16_t s[ADAMW_LDS];
  const lora_adamw_tile tile = p.tiles[blockIdx.x];
  const lora_adamw_tensor& t = tile.tensor;
  // the whole record is here before anything is decided by it: read field by field where each is
  // needed, it costs a round of latency each
  asm volatile("" ::"s"(t.param), "s"(t.grad), "s"(t.m), "s"(t.v), "s"(t.m_scale), "s"(t.v_scale), "s"(t.copy), "s"(t.pack),
               "s"(t.pack_bwd), "s"(t.rows), "s"(t.cols), "s"(t.group), "s"(t.kind), "s"(tile.first));
  c_float* cp = (c_float*)(reinterpret_cast<uintptr_t>(p.coef) + (size_t)t.group * ADAMW_COEF * sizeof(float));
  if (ALONE ? p.active && !p.active[t.group] : cp[9] == 0.f) return;
  const Place at = place(t, tile.first);
  // The tile in LDS: A's rows padded so that eight rows' columns lie in other banks (by 4 where a quad
  // lies in one row, and else to an odd length), B's by 8, which keeps its 16-byte pieces aligned.
  const bool pack_a = t.kind == KIND_A && (t.pack || t.pack_bwd), pack_b = t.kind == KIND_B && (t.pack || t.pack_bwd);
  const int ld = t.kind == KIND_A ? (t.cols % 4 == 0 ? t.cols + 4 : t.cols | 1) : 4 * at.len4 + 8;
  __shared__ float shared_coef[ADAMW_COEF];
  int step = 0;
  auto coef = [&]() {
    if (!ALONE) return get(cp);
    if (threadIdx.x < 64) {  // one wave for all: 64-bit arithmetic of all waves would take longer than the loads
      step = p.steps[t.group] + 1;
      const Coef c = coefficients(p.hyper + (long)t.group * ADAMW_HYPER, step, 1.0);
      if (threadIdx.x == 0) put(shared_coef, c, true);
    }
    __syncthreads();
    return get(shared_coef);
  };
  if (at.n % ADAMW_BLOCK) update<BITS8, CLIP, PAST, WG, true>(t, at, s, ld, pack_a, pack_b, coef);
  else update<BITS8, CLIP, PAST, WG, false>(t, at, s, ld, pack_a, pack_b, coef);
  if (ALONE && threadIdx.x == 0) {  // this workgroup has read the group's step
    if (add_agent(p.arrived + ADAMW_LINE * t.group, 1) == p.group_first[t.group + 1] - p.group_first[t.group] - 1) {
      p.steps[t.group] = step;
      set_agent(p.arrived + ADAMW_LINE * t.group, 0);
    }
  }
  if (pack_a || pack_b) __syncthreads();
  if (pack_a) write_packs_a<WG>(s, ld, t.cols, tile.first, at.n / t.cols, t.rows, t.pack, t.cols % 8 ? t.pack_bwd : nullptr);
  if (pack_b) write_packs_b<WG>(s, ld, t.rows, tile.first, 4 * at.len4, t.cols, t.pack_bwd, t.pack);
}

// Steps of few tiles without norms are one launch.  Each arrival at a group's counter takes about 13 ns,
// one behind another where all tiles are one group's, and goes on beside the other tiles' work: 80 tiles
// 6.8 us with a launch for the groups, 6.1 without; 304 in 8 bits 13.0 and 12.0; 992 of one group 28.4
// and 28.4; 816 of small tiles 18.3 and 18.7 (about even from 800 tiles on).
constexpr long ALONE_TILES = 1024;

// With norms, the groups of so few tiles are settled in the norms' launch by the same arrivals (32 tiles
// 11.7 us with a launch for the groups, 9.6 without; 80 12.0 and 10.9; 304 of one group 17.0 and 19.5).
// What makes it slower is many arrivals at one group's counter: the rule counts all tiles, as if they were
// one group's, and where they are many groups' it gives up its gain sooner than it would have to.
constexpr long LAST_TILES = 128;

// Steps of more tiles than this read and write their states and master copies past the caches, which
// could not hold them until the next step: what the norms' launch has read of the gradients then stays
// for the update (the layer above: 265 us within them, 237 past them, with norms).  Codes and scales of
// 8-bit states stay within: a wave's 256 bytes are too short for it (188 us with all within the caches,
// 180 with the master copies past them, 190 with all).  Full tiles, as many as this, are
// 8 million values: about 185 MB with gradients and packed forms, 135 in 8 bits.  Tiles of small ranks hold
// fewer (512 values of rank 1), and a step of theirs would fit the caches.  With other work between two
// steps (1 GiB copied before each) it is the same to them: 32 tenants of rank 1 without norms 51 us past the
// caches and 51 within, in 8 bits 55 and 55, of rank 4 69 and 69 (63 and 63).  Steps one right behind another
// lose by it: 48 and 40 us of rank 1, 50 and 43 in 8 bits; of rank 8 in 8 bits (8.9 million values) 52 and 47.
constexpr long STREAM_TILES = 2048;

constexpr int WG = 1024;

template <bool BITS8>
void launch_update(const AdamWParams& p, bool alone, hipStream_t s) {
  const dim3 grid((unsigned)p.n_tiles), wg(WG);
  const bool past = p.n_tiles > STREAM_TILES;
  if (alone) hipLaunchKernelGGL((k_adamw<BITS8, false, true, false, WG>), grid, wg, 0, s, p);
  else if (p.norm && past) hipLaunchKernelGGL((k_adamw<BITS8, true, false, true, WG>), grid, wg, 0, s, p);
  else if (p.norm) hipLaunchKernelGGL((k_adamw<BITS8, true, false, false, WG>), grid, wg, 0, s, p);
  else if (past) hipLaunchKernelGGL((k_adamw<BITS8, false, false, true, WG>), grid, wg, 0, s, p);
  else hipLaunchKernelGGL((k_adamw<BITS8, false, false, false, WG>), grid, wg, 0, s, p);
}

}  // namespace

hipError_t launch_adamw(const AdamWParams& p, int state_bits, hipStream_t s) {
  const bool alone = !p.norm && p.n_tiles <= ALONE_TILES, last = p.norm && p.n_tiles <= LAST_TILES;
  const unsigned norm_wgs = (unsigned)((p.n_tiles + 3) / 4);
  if (last) hipLaunchKernelGGL(k_adamw_norms<true>, dim3(norm_wgs + (p.n_groups + 255) / 256), dim3(256), 0, s, p);
  else if (p.norm) hipLaunchKernelGGL(k_adamw_norms<false>, dim3(norm_wgs), dim3(256), 0, s, p);
  if (!alone && !last) hipLaunchKernelGGL(k_adamw_groups, dim3(p.n_groups), dim3(256), 0, s, p);
  if (p.n_tiles == 0) return hipGetLastError();
  if (state_bits == 8) launch_update<true>(p, alone, s);
  else launch_update<false>(p, alone, s);
  return hipGetLastError();
}

}  // namespace lora
