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
// so its loads and stores run over whole cache lines.
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

// One wave takes `per_wave` rounds of a token: a round is 64 / LPH heads of one kind (queries,
// keys or, for the append, values).  The loads of all its rounds are issued before the first
// is used.
template <int D, int MODE, int PW>
__global__ __launch_bounds__(256) void k_norm_rope(RopeParams p) {
  constexpr int LPH = D / 16, SLOTS = 64 / LPH;
  const int lane = threadIdx.x & 63;
  const int item = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  const int t = item / p.groups;
  if (t >= p.T) return;
  const int r0 = (item - t * p.groups) * PW;
  const int rounds = p.rounds_q + p.rounds_k + (MODE == FORWARD ? 0 : p.rounds_v);
  const int sl = lane / LPH, j = lane % LPH;
  const LaneMap m = lane_map(j, p.rot, p.interleaved);

  uint4 xa[PW], xb[PW];
#pragma unroll
  for (int i = 0; i < PW; ++i) {
    const int r = r0 + i;
    xa[i] = xb[i] = zero4();
    if (r >= rounds) continue;
    const int kind = r < p.rounds_q ? 0 : r < p.rounds_q + p.rounds_k ? 1 : 2;
    const int h = (r - (kind == 0 ? 0 : kind == 1 ? p.rounds_q : p.rounds_q + p.rounds_k)) * SLOTS + sl;
    if (h >= (kind == 0 ? p.n_q : p.n_kv)) continue;
    const uint16_t* src = p.qkv + (long)t * p.ld + (long)(h + (kind == 0 ? 0 : kind == 1 ? p.n_q : p.n_q + p.n_kv)) * D;
    xa[i] = ldg16(src + m.a);
    xb[i] = ldg16(src + m.b);
  }
  int pos = p.rot ? p.positions[t] : 0;
  const bool placed = p.rot == 0 || (unsigned)pos < (unsigned)p.max_pos;
  if (!placed) {
    pos = 0;
    if (p.status && lane == 0 && r0 == 0) or_agent(p.status, ST_POSITION);
  }
  int slot = 0;
  if (MODE != FORWARD) {
    slot = p.slots[t];
    if ((long)slot >= p.n_slots) {
      slot = -1;
      if (p.status && lane == 0 && r0 == 0) or_agent(p.status, ST_SLOT);
    }
    if (!placed) slot = -1;
  }
  const Turn tn = load_turn(p.cos_sin, pos, p.rot, m);

#pragma unroll
  for (int i = 0; i < PW; ++i) {
    const int r = r0 + i;
    if (r >= rounds) break;
    const int kind = r < p.rounds_q ? 0 : r < p.rounds_q + p.rounds_k ? 1 : 2;
    const int h = (r - (kind == 0 ? 0 : kind == 1 ? p.rounds_q : p.rounds_q + p.rounds_k)) * SLOTS + sl;
    const bool live = h < (kind == 0 ? p.n_q : p.n_kv);
    float v[16];
    widen(xa[i], v);
    widen(xb[i], v + 8);
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
    if (!live) continue;
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
}

// Backward.  Waves stride over the tokens; a lane meets the same 16 places of the head in
// every round, so the weights' gradients grow in its registers and are joined at the end:
// over the wave's slots and the workgroup's waves in LDS, in a fixed order, into one row of
// partial sums a workgroup, which k_weight_grad adds in order (no atomics: the result does
// not depend on timing).
template <int D>
__global__ __launch_bounds__(256) void k_norm_rope_bwd(RopeBwdParams p) {
  constexpr int LPH = D / 16, SLOTS = 64 / LPH, ROWS = 4 * SLOTS;
  __shared__ __attribute__((aligned(16))) float red[ROWS][2 * D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sl = lane / LPH, j = lane % LPH;
  const LaneMap m = lane_map(j, p.rot, p.interleaved);
  const int rounds = p.rounds_q + p.rounds_k + p.rounds_v;
  float accq[16], acck[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) accq[e] = acck[e] = 0.f;

  for (int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + wave)); t < p.T; t += p.n_wg * 4) {
    int pos = p.rot ? p.positions[t] : 0;
    const bool placed = p.rot == 0 || (unsigned)pos < (unsigned)p.max_pos;
    if (!placed) {
      pos = 0;
      if (p.status && lane == 0) or_agent(p.status, ST_POSITION);
    }
    const Turn tn = load_turn(p.cos_sin, pos, p.rot, m);
    for (int r = 0; r < rounds; ++r) {
      const int kind = r < p.rounds_q ? 0 : r < p.rounds_q + p.rounds_k ? 1 : 2;
      const int h = (r - (kind == 0 ? 0 : kind == 1 ? p.rounds_q : p.rounds_q + p.rounds_k)) * SLOTS + sl;
      const bool live = h < (kind == 0 ? p.n_q : p.n_kv);
      const long col = (long)(h + (kind == 0 ? 0 : kind == 1 ? p.n_q : p.n_q + p.n_kv)) * D;
      const uint16_t* gsrc = kind == 0 ? p.dq + ((long)t * p.n_q + h) * D
                                       : (kind == 1 ? p.dk : p.dv) + ((long)t * p.n_kv + h) * D;
      uint16_t* dst = p.dqkv + (long)t * p.ldd + col;
      uint4 ga = zero4(), gb = zero4(), xa = zero4(), xb = zero4();
      if (live) {
        ga = ldg16(gsrc + m.a);
        gb = ldg16(gsrc + m.b);
      }
      if (kind == 2) {  // values pass through
        if (live) {
          *reinterpret_cast<uint4*>(dst + m.a) = ga;
          *reinterpret_cast<uint4*>(dst + m.b) = gb;
        }
        continue;
      }
      const float* w = kind == 0 ? p.q_weight : p.k_weight;
      if (live && w) {
        const uint16_t* src = p.qkv + (long)t * p.ld + col;
        xa = ldg16(src + m.a);
        xb = ldg16(src + m.b);
      }
      float g[16];
      widen(ga, g);
      widen(gb, g + 8);
      turn<-1>(g, tn, p.interleaved, m.turns);
      if (w) {
        float x[16];
        widen(xa, x);
        widen(xb, x + 8);
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
            const float d = count ? g[e] * x[e] : 0.f;
            if (kind == 0) accq[e] += d; else acck[e] += d;
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
  }
  if (!p.q_weight) return;
  float* row = red[wave * SLOTS + sl];
#pragma unroll
  for (int q4 = 0; q4 < 4; ++q4) {
    const int o = (q4 < 2 ? m.a : m.b - 8) + 4 * q4;
    *reinterpret_cast<float4*>(row + o) = make_float4(accq[4 * q4], accq[4 * q4 + 1], accq[4 * q4 + 2], accq[4 * q4 + 3]);
    *reinterpret_cast<float4*>(row + D + o) = make_float4(acck[4 * q4], acck[4 * q4 + 1], acck[4 * q4 + 2], acck[4 * q4 + 3]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += 256) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) v += red[i][c];
    p.part[(long)blockIdx.x * 2 * D + c] = v;
  }
}

// dw[c] = sum over the workgroups' rows, 16 columns a workgroup: 64 threads a float4 column
// stride over the rows, then add up in LDS, all in a fixed order.
__global__ __launch_bounds__(256) void k_weight_grad(const float* __restrict__ part, int n, int D, float* dqw, float* dkw) {
  __shared__ float4 red[64][4];
  const int c4 = threadIdx.x & 3, rg = threadIdx.x >> 2;
  const int col = blockIdx.x * 16 + 4 * c4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int r = rg; r < n; r += 64) {
    const float4 u = *reinterpret_cast<const float4*>(part + (long)r * 2 * D + col);
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  red[rg][c4] = v;
  __syncthreads();
  for (int s = 32; s >= 1; s >>= 1) {
    if (rg < s) {
      const float4 u = red[rg + s][c4];
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      red[rg][c4] = v;
    }
    __syncthreads();
  }
  if (rg == 0) *reinterpret_cast<float4*>(col < D ? dqw + col : dkw + col - D) = v;
}

template <int D, int MODE>
hipError_t launch_mode(RopeParams p, hipStream_t s) {
  constexpr int SLOTS = 64 / (D / 16);
  p.rounds_q = (p.n_q + SLOTS - 1) / SLOTS;
  p.rounds_k = (p.n_kv + SLOTS - 1) / SLOTS;
  p.rounds_v = MODE == FORWARD ? 0 : p.rounds_k;
  const int rounds = p.rounds_q + p.rounds_k + p.rounds_v;
  const bool wide = (long)p.T * rounds >= 4096;
  p.per_wave = wide ? 4 : 1;
  p.groups = (rounds + p.per_wave - 1) / p.per_wave;
  const dim3 grid((unsigned)(((long)p.T * p.groups + 3) / 4));
  if (wide)
    hipLaunchKernelGGL((k_norm_rope<D, MODE, 4>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((k_norm_rope<D, MODE, 1>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int D>
hipError_t launch_bwd(RopeBwdParams p, hipStream_t s) {
  constexpr int SLOTS = 64 / (D / 16);
  p.rounds_q = (p.n_q + SLOTS - 1) / SLOTS;
  p.rounds_k = (p.n_kv + SLOTS - 1) / SLOTS;
  p.rounds_v = p.dv ? p.rounds_k : 0;
  if (p.T > 0) hipLaunchKernelGGL(k_norm_rope_bwd<D>, dim3(p.n_wg), dim3(256), 0, s, p);
  if (p.q_weight)
    hipLaunchKernelGGL(k_weight_grad, dim3(2 * D / 16), dim3(256), 0, s, p.part, p.n_wg, D, p.dqw, p.dkw);
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
