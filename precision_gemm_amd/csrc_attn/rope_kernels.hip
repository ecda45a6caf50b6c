// Norms of the query and key heads with the position rotation in the same pass: forward,
// backward, and on the way into a paged cache.
//
// Mathematics, for one head x of D values at position p (c, s: row p of the table):
//   n_d = x_d r w_d,  r = 1 / sqrt(mean(x^2) + eps);    without weights n = x
//   y_a = n_a c_i - n_b s_i,  y_b = n_b c_i + n_a s_i   for each rotated pair (a, b)
// and backwards, with g the rotation by -p of dy and xh = x r:
//   dw_d += g_d xh_d,  dx = r (g w - xh mean(g w xh)).
//
// All three are bound by HBM (about 10 operations a value).  Lane layout: D / 16 lanes share
// a head, and a lane holds two 16-byte chunks of it that contain both members of every pair
// it rotates, so the rotation needs no exchange between lanes, whichever way the pairs are
// laid out and however much of the head is rotated; only the norm's sums cross lanes
// (log2(D / 16) butterfly steps).  The 64 / (D / 16) heads of a wave's round are neighbours,
// so its loads and stores run over whole cache lines.  Results are stored the ordinary way:
// stores past the caches make these kernels faster alone (4,096 tokens, backward: 33.9 to 29.3 us)
// and whoever reads the results slower by more (with a copy of them 48.8 to 52.2 us).
#include <algorithm>

#include "attn_kernels.hpp"
#include "../csrc/device_common.hpp"

namespace lora {
namespace {

constexpr int ST_POSITION = 1, ST_SLOT = 2;  // LORA_ATTN_BAD_POSITION, LORA_ATTN_BAD_SLOT

// The two chunks of lane j of a head, and its places in the table's row.
struct LaneMap {
  int a, b;       // element offsets of the chunks
  int t0, t1;     // table offsets of the lane's first and last four cosines
  bool turns;     // the lane's chunks are rotated
};

__device__ __forceinline__ LaneMap lane_map(int j, int rot, int interleaved) {
  const int nr = rot >> 4;  // lanes whose chunks are rotated
  LaneMap m;
  m.turns = j < nr;
  const int ca = m.turns ? j : 2 * nr + 2 * (j - nr);
  const int cb = m.turns ? j + nr : ca + 1;
  m.a = 8 * ca;
  m.b = 8 * cb;
  m.t0 = interleaved ? 4 * ca : 8 * j;
  m.t1 = interleaved ? 4 * cb : 8 * j + 4;
  return m;
}

struct Turn { float c[8], s[8]; };

// Row `pos` of the table for this lane; the identity where the lane's chunks do not turn.
__device__ __forceinline__ Turn load_turn(const float* cos_sin, int pos, int rot, const LaneMap& m) {
  Turn t;
#pragma unroll
  for (int e = 0; e < 8; ++e) { t.c[e] = 1.f; t.s[e] = 0.f; }
  if (m.turns) {
    const float* row = cos_sin + (long)pos * rot;
    const float4 c0 = *reinterpret_cast<const float4*>(row + m.t0), c1 = *reinterpret_cast<const float4*>(row + m.t1);
    const float* sr = row + (rot >> 1);
    const float4 s0 = *reinterpret_cast<const float4*>(sr + m.t0), s1 = *reinterpret_cast<const float4*>(sr + m.t1);
    t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w; t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
    t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w; t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
  }
  return t;
}

// Turn the 16 values of a lane (chunk a in v[0..7], chunk b in v[8..15]); SIGN -1 turns back.
template <int SIGN>
__device__ __forceinline__ void turn(float (&v)[16], const Turn& t, int interleaved, bool turns) {
  if (!turns) return;  // not 1 * x - 0 * y: an infinite y would make that NaN
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = v[2 * e], b = v[2 * e + 1], s = SIGN * t.s[e];
      v[2 * e] = a * t.c[e] - b * s;
      v[2 * e + 1] = b * t.c[e] + a * s;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = v[e], b = v[8 + e], s = SIGN * t.s[e];
      v[e] = a * t.c[e] - b * s;
      v[8 + e] = b * t.c[e] + a * s;
    }
  }
}

__device__ __forceinline__ void widen(const uint4& w, float* v) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 narrow(const float* v) {
  return make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
}

// Sum over the LPH neighbouring lanes of a head.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int d = 1; d < LPH; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// e4m3 code of x: nearest even, saturated at +-448, NaN kept (a plain clamp would drop it).
__device__ __forceinline__ float sat448(float x) { return x != x ? x : fminf(fmaxf(x, -448.f), 448.f); }
__device__ __forceinline__ uint32_t fp8x4(const float* v) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(sat448(v[0]), sat448(v[1]), r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(sat448(v[2]), sat448(v[3]), r, true);
  return (uint32_t)r;
}

enum { FORWARD = 0, APPEND_BF16 = 1, APPEND_FP8 = 2 };

// A wave takes one round of a token: 64 / LPH heads of one kind (queries, keys or, for the append,
// values).  Waves this short hide each other's latencies; two, three and four rounds a wave, all
// loads first, are slower up to 1,024 tokens (32 + 8 + 8 heads of 128, 16 tokens: 3.0 us, then 3.8,
// 4.6 and 5.4) and no faster at 4,096 (21.7 us with inputs out of HBM, 4.0 TB/s; 22.6, 23.0, 23.9;
// a copy of as many bytes 19.3).
template <int D, int MODE>
__global__ __launch_bounds__(256) void k_norm_rope(RopeParams p) {
  constexpr int LPH = D / 16, SLOTS = 64 / LPH;
  const int lane = threadIdx.x & 63;
  const int item = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  const int rounds = p.rounds_q + p.rounds_k + (MODE == FORWARD ? 0 : p.rounds_k);
  const int t = item / rounds, r = item - t * rounds;
  if (t >= p.T) return;
  const int sl = lane / LPH, j = lane % LPH;
  const LaneMap m = lane_map(j, p.rot, p.interleaved);

  const int kind = r < p.rounds_q ? 0 : r < p.rounds_q + p.rounds_k ? 1 : 2;
  const int h = (r - (kind == 0 ? 0 : kind == 1 ? p.rounds_q : p.rounds_q + p.rounds_k)) * SLOTS + sl;
  const bool live = h < (kind == 0 ? p.n_q : p.n_kv);
  uint4 xa = zero4(), xb = zero4();
  if (live) {
    const uint16_t* src = p.qkv + (long)t * p.ld + (long)(h + (kind == 0 ? 0 : kind == 1 ? p.n_q : p.n_q + p.n_kv)) * D;
    xa = ldg16(src + m.a);
    xb = ldg16(src + m.b);
  }
  int pos = p.rot ? p.positions[t] : 0;
  const bool placed = p.rot == 0 || (unsigned)pos < (unsigned)p.max_pos;
  if (!placed) {
    pos = 0;
    if (p.status && lane == 0 && r == 0) or_agent(p.status, ST_POSITION);
  }
  int slot = 0;
  if (MODE != FORWARD) {
    slot = p.slots[t];
    if ((long)slot >= p.n_slots) {
      slot = -1;
      if (p.status && lane == 0 && r == 0) or_agent(p.status, ST_SLOT);
    }
    if (!placed) slot = -1;
  }
  const Turn tn = load_turn(p.cos_sin, pos, p.rot, m);

  float v[16];
  widen(xa, v);
  widen(xb, v + 8);
  if (MODE == FORWARD || kind < 2) {
    const float* w = kind == 0 ? p.q_weight : p.k_weight;
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss += v[e] * v[e];
      const float rs = 1.0f / sqrtf(head_sum<LPH>(ss) * (1.0f / D) + p.eps);
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        const float4 w4 = *reinterpret_cast<const float4*>(w + (q4 < 2 ? m.a : m.b - 8) + 4 * q4);
        v[4 * q4] *= rs * w4.x; v[4 * q4 + 1] *= rs * w4.y; v[4 * q4 + 2] *= rs * w4.z; v[4 * q4 + 3] *= rs * w4.w;
      }
    }
    turn<1>(v, tn, p.interleaved, m.turns);
  }
  if (!live) return;
  if (MODE == FORWARD || kind == 0) {
    uint16_t* dst = kind == 0 ? p.q_out + (long)t * p.ldq + (long)h * D : p.k_out + (long)t * p.ldk + (long)h * D;
    *reinterpret_cast<uint4*>(dst + m.a) = placed ? narrow(v) : zero4();
    *reinterpret_cast<uint4*>(dst + m.b) = placed ? narrow(v + 8) : zero4();
  } else if (slot >= 0) {
    const int off = slot & ((1 << p.page_log2) - 1);
    const long row = ((((long)(slot >> p.page_log2) * p.n_kv + h) << p.page_log2) + off) * D;
    if (MODE == APPEND_BF16) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(kind == 1 ? p.k_cache : p.v_cache) + row;
      *reinterpret_cast<uint4*>(dst + m.a) = narrow(v);
      *reinterpret_cast<uint4*>(dst + m.b) = narrow(v + 8);
    } else {
      uint8_t* dst = reinterpret_cast<uint8_t*>(kind == 1 ? p.k_cache : p.v_cache) + row;
      const float inv = 1.0f / (kind == 1 ? p.k_scale : p.v_scale)[h];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= inv;
      *reinterpret_cast<uint2*>(dst + m.a) = make_uint2(fp8x4(v), fp8x4(v + 4));
      *reinterpret_cast<uint2*>(dst + m.b) = make_uint2(fp8x4(v + 8), fp8x4(v + 12));
    }
  }
}

// Backward.  A workgroup takes query heads (the first q_wg workgroups) or key and value heads,
// so that a lane, which meets the same 16 places of the head in every round, needs one set of
// sums for the weights' gradient; a wave takes an equal, contiguous share of the (token, round)
// pairs of its kind, the next round's loads in flight while one is computed.  The sums are
// joined over the wave's slots and the workgroup's waves in LDS, in a fixed order, into one row
// a workgroup, which k_weight_grad adds in order (no atomics: the result does not depend on
// timing).  4,096 tokens of 32 + 8 + 8 heads of 128 (145 MB): 31.9 us, 4.5 TB/s; 512 workgroups
// instead of 768 take 8 % longer, 256 55 %; two rounds in flight instead of one 3 %.
template <int D>
__global__ __launch_bounds__(256, 3) void k_norm_rope_bwd(RopeBwdParams p) {
  constexpr int LPH = D / 16, SLOTS = 64 / LPH, ROWS = 4 * SLOTS;
  __shared__ __attribute__((aligned(16))) float red[ROWS][D];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int sl = lane / LPH, j = lane % LPH;
  const LaneMap m = lane_map(j, p.rot, p.interleaved);
  const bool kv = (int)blockIdx.x >= p.q_wg;
  const int rounds = kv ? 2 * p.rounds_k : p.rounds_q;  // values' rounds too, without dv empty
  const float* w = kv ? p.k_weight : p.q_weight;
  const int n_waves = 4 * (kv ? p.n_wg - p.q_wg : p.q_wg), at = 4 * ((int)blockIdx.x - (kv ? p.q_wg : 0)) + wave;
  const int all = p.T * rounds;
  const int first = (int)((long)all * at / n_waves), last = (int)((long)all * (at + 1) / n_waves);

  // a (token, round): heads h of this lane's slot, places of its gradient, input and result
  struct Round { uint4 ga, gb, xa, xb; };
  auto head = [&](int r, bool& value, bool& live) {
    value = kv && r >= p.rounds_k;
    const int h = (value ? r - p.rounds_k : r) * SLOTS + sl;
    live = h < (kv ? p.n_kv : p.n_q) && !(value && !p.dv);
    return h;
  };
  auto load = [&](int t, int r) {
    bool value, live;
    const int h = head(r, value, live);
    const uint16_t* g = (kv ? (value ? p.dv : p.dk) + ((long)t * p.n_kv + h) * D : p.dq + ((long)t * p.n_q + h) * D);
    const uint16_t* x = p.qkv + (long)t * p.ld + (long)(h + (kv ? p.n_q : 0)) * D;
    Round v{zero4(), zero4(), zero4(), zero4()};
    if (live) {
      v.ga = ldg16(g + m.a);
      v.gb = ldg16(g + m.b);
      if (w && !value) {
        v.xa = ldg16(x + m.a);
        v.xb = ldg16(x + m.b);
      }
    }
    return v;
  };

  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  int t = first / rounds, r = first - t * rounds;
  Round next{};
  if (first < last) next = load(t, r);
  bool placed = true, fresh = true;
  Turn tn;
  for (int it = first; it < last; ++it) {
    const Round now = next;
    const int t0 = t, r0 = r;
    if (fresh) {  // a token's first round here
      int pos = p.rot ? p.positions[t0] : 0;
      placed = p.rot == 0 || (unsigned)pos < (unsigned)p.max_pos;
      if (!placed) {
        pos = 0;
        if (p.status && lane == 0) or_agent(p.status, ST_POSITION);
      }
      tn = load_turn(p.cos_sin, pos, p.rot, m);
    }
    fresh = ++r == rounds;
    if (fresh) {
      r = 0;
      ++t;
    }
    if (it + 1 < last) next = load(t, r);

    bool value, live;
    const int h = head(r0, value, live);
    uint16_t* dst = p.dqkv + (long)t0 * p.ldd + (long)(h + (kv ? (value ? p.n_q + p.n_kv : p.n_q) : 0)) * D;
    if (value) {  // values pass through
      if (live) {
        *reinterpret_cast<uint4*>(dst + m.a) = now.ga;
        *reinterpret_cast<uint4*>(dst + m.b) = now.gb;
      }
      continue;
    }
    float g[16];
    widen(now.ga, g);
    widen(now.gb, g + 8);
    turn<-1>(g, tn, p.interleaved, m.turns);
    if (w) {
      float x[16];
      widen(now.xa, x);
      widen(now.xb, x + 8);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss += x[e] * x[e];
      const float rs = 1.0f / sqrtf(head_sum<LPH>(ss) * (1.0f / D) + p.eps);
      float dot = 0.f;
      const bool count = live && placed;
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        const float4 w4 = *reinterpret_cast<const float4*>(w + (q4 < 2 ? m.a : m.b - 8) + 4 * q4);
        const float ww[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * q4 + i;
          x[e] *= rs;                       // xh
          acc[e] += count ? g[e] * x[e] : 0.f;
          g[e] *= ww[i];
          dot += g[e] * x[e];
        }
      }
      const float mean = head_sum<LPH>(dot) * (1.0f / D);
#pragma unroll
      for (int e = 0; e < 16; ++e) g[e] = rs * (g[e] - x[e] * mean);
    }
    if (live) {
      *reinterpret_cast<uint4*>(dst + m.a) = placed ? narrow(g) : zero4();
      *reinterpret_cast<uint4*>(dst + m.b) = placed ? narrow(g + 8) : zero4();
    }
  }
  if (!w) return;
  float* row = red[wave * SLOTS + sl];
#pragma unroll
  for (int q4 = 0; q4 < 4; ++q4)
    *reinterpret_cast<float4*>(row + (q4 < 2 ? m.a : m.b - 8) + 4 * q4) = make_float4(acc[4 * q4], acc[4 * q4 + 1], acc[4 * q4 + 2], acc[4 * q4 + 3]);
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += 256) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) v += red[i][c];
    p.part[(long)blockIdx.x * D + c] = v;
  }
}

// dw[c] = sum over the workgroups' rows of its kind, 16 columns a workgroup: 256 threads a
// float4 column stride over the rows, then add up in a fixed order.  768 rows of 128: 4.6 us, a
// launch and three rounds of loads.
__global__ __launch_bounds__(1024) void k_weight_grad(const float* __restrict__ part, int q_wg, int n_wg, int D, float* dqw, float* dkw) {
  __shared__ float4 red[16][4];
  const int c4 = threadIdx.x & 3, rg = threadIdx.x >> 2;
  const int blocks = D / 16;
  const bool k = (int)blockIdx.x >= blocks;
  const int col = (blockIdx.x - (k ? blocks : 0)) * 16 + 4 * c4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int r = (k ? q_wg : 0) + rg; r < (k ? n_wg : q_wg); r += 256) {
    const float4 u = *reinterpret_cast<const float4*>(part + (long)r * D + col);
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
#pragma unroll
  for (int d = 4; d < 64; d <<= 1) {
    v.x += __shfl_xor(v.x, d); v.y += __shfl_xor(v.y, d); v.z += __shfl_xor(v.z, d); v.w += __shfl_xor(v.w, d);
  }
  if ((threadIdx.x & 63) < 4) red[threadIdx.x >> 6][c4] = v;
  __syncthreads();
  if (rg) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) {
    const float4 u = red[w][c4];
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  *reinterpret_cast<float4*>((k ? dkw : dqw) + col) = v;
}

template <int D, int MODE>
hipError_t launch_mode(RopeParams p, hipStream_t s) {
  constexpr int SLOTS = 64 / (D / 16);
  p.rounds_q = (p.n_q + SLOTS - 1) / SLOTS;
  p.rounds_k = (p.n_kv + SLOTS - 1) / SLOTS;
  const int rounds = p.rounds_q + p.rounds_k + (MODE == FORWARD ? 0 : p.rounds_k);
  hipLaunchKernelGGL((k_norm_rope<D, MODE>), dim3((unsigned)(((long)p.T * rounds + 3) / 4)), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int D>
hipError_t launch_bwd(RopeBwdParams p, hipStream_t s) {
  constexpr int SLOTS = 64 / (D / 16);
  p.rounds_q = (p.n_q + SLOTS - 1) / SLOTS;
  p.rounds_k = (p.n_kv + SLOTS - 1) / SLOTS;
  // workgroups of each kind by its rounds, a wave a round at least (the split, and with it the
  // order of the sums, does not depend on whether dv is given)
  const int rounds = p.rounds_q + 2 * p.rounds_k;
  p.q_wg = (int)std::min<long>(std::max(1, ROPE_BWD_WGS * p.rounds_q / rounds), ((long)p.T * p.rounds_q + 3) / 4);
  p.n_wg = p.q_wg + (int)std::min<long>(ROPE_BWD_WGS - ROPE_BWD_WGS * p.rounds_q / rounds, ((long)p.T * 2 * p.rounds_k + 3) / 4);
  if (p.T > 0) hipLaunchKernelGGL(k_norm_rope_bwd<D>, dim3(p.n_wg), dim3(256), 0, s, p);
  if (p.q_weight)
    hipLaunchKernelGGL(k_weight_grad, dim3(2 * D / 16), dim3(1024), 0, s, p.part, p.q_wg, p.n_wg, D, p.dqw, p.dkw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_rope(const RopeParams& p, int D, hipStream_t s) {
  switch (D) {
    case 64: return launch_mode<64, FORWARD>(p, s);
    case 128: return launch_mode<128, FORWARD>(p, s);
    default: return launch_mode<256, FORWARD>(p, s);
  }
}

hipError_t launch_rope_append(const RopeParams& p, int D, bool fp8, hipStream_t s) {
  switch (D) {
    case 64: return fp8 ? launch_mode<64, APPEND_FP8>(p, s) : launch_mode<64, APPEND_BF16>(p, s);
    case 128: return fp8 ? launch_mode<128, APPEND_FP8>(p, s) : launch_mode<128, APPEND_BF16>(p, s);
    default: return fp8 ? launch_mode<256, APPEND_FP8>(p, s) : launch_mode<256, APPEND_BF16>(p, s);
  }
}

hipError_t launch_norm_rope_bwd(const RopeBwdParams& p, int D, hipStream_t s) {
  switch (D) {
    case 64: return launch_bwd<64>(p, s);
    case 128: return launch_bwd<128>(p, s);
    default: return launch_bwd<256>(p, s);
  }
}

}  // namespace lora
