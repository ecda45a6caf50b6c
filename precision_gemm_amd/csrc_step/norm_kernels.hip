// Layer norm and RMS norm of rows of hidden states, forward (with the residual's addition) and
// backward.
//
// Mathematics, for one row h of K values (mu = 0 for the RMS norm):
//   mu = mean(h),  r = 1 / sqrt(mean((h - mu)^2) + eps),  xh = (h - mu) r,  y = xh w + b
// and backwards, with g = dy w:
//   dh = r (g - mean(g) - xh mean(g xh))   (without mean(g) for the RMS norm)
//   dw = sum over the rows of dy xh,  db = sum of dy.
#include <algorithm>

#include "step_kernels.hpp"
#include "../csrc/device_common.hpp"

namespace lora {
namespace {

__device__ __forceinline__ void widen(const uint4& w, float* v) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 narrow(const float* v) {
  return make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
}
__device__ __forceinline__ void ld8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// The compiler takes the value as new from here on.
__device__ __forceinline__ void opaque(uint4& v) { asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w)); }

// Sum over a wave, the same in every lane: four steps within rows of 16 lanes, two across them,
// on the DPP path (no LDS).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xf>(v);  // from 1, 2, 4 and 8 lanes below
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);  // lane 15 of a row to the next (rows 1 and 3)
  v = dpp_add<0x143, 0xc>(v);  // lane 31 to the upper half
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Sums over the WAVES neighbouring waves that share a row; `slot` is LDS of this sum alone.
template <int WAVES, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*slot)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (WAVES == 1) return;
  const int wave = threadIdx.x >> 6, first = wave / WAVES * WAVES;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) slot[wave][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += slot[first + w][i];
    v[i] = s;
  }
}

// TPR threads a row, C chunks of 8 values a thread, WG threads a workgroup.
template <int TPR, int C, int WG, bool RMS>
__global__ __launch_bounds__(WG) void k_norm(NormParams p) {
  constexpr int WAVES = TPR / 64;
  __shared__ float red[2][WG / 64][1];
  const int tid = threadIdx.x % TPR;
  const int t = blockIdx.x * (WG / TPR) + threadIdx.x / TPR;
  const bool row = t < p.T;
  float h[C][8];
  bool live[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TPR + tid) * 8;
    live[c] = row && col < p.K;
    uint4 a = zero4();
    if (live[c]) a = ldg16(p.x + (long)t * p.ldx + col);
    widen(a, h[c]);
  }
  if (p.residual) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TPR + tid) * 8;
      uint4 a = zero4();
      if (live[c]) a = ldg16(p.residual + (long)t * p.ldr + col);
      float r[8];
      widen(a, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] += h[c][e];
      a = narrow(r);  // the stream's own rounding: the statistics are those of what is stored
      if (live[c]) *reinterpret_cast<uint4*>(p.sum + (long)t * p.lds + col) = a;
      widen(a, h[c]);
    }
  }
  float mean = 0.f;
  if (!RMS) {
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += h[c][e];
    row_sum<WAVES, 1>(s, red[0]);
    mean = s[0] / (float)p.K;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[c][e] -= mean;
      q[0] += live[c] ? h[c][e] * h[c][e] : 0.f;
    }
  row_sum<WAVES, 1>(q, red[1]);
  const float r = 1.0f / sqrtf(q[0] / (float)p.K + p.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TPR + tid) * 8;
    if (!live[c]) continue;
    float w[8], b[8];
    if (p.weight) ld8(p.weight + col, w);
    if (p.bias) ld8(p.bias + col, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = h[c][e] * r;
      if (p.weight) v *= w[e];
      if (p.bias) v += b[e];
      h[c][e] = v;
    }
    *reinterpret_cast<uint4*>(p.y + (long)t * p.ldy + col) = narrow(h[c]);
  }
}

// Backward.  A workgroup takes rows blockIdx.x * (WG / TPR) + ... in strides of the grid; a
// thread meets the same columns in every row, so it keeps their sums for the weights' gradients
// in registers.
template <int TPR, int C, int WG, bool AHEAD, bool RMS>
__global__ __launch_bounds__(WG) void k_norm_bwd(NormBwdParams p) {
  constexpr int WAVES = TPR / 64, ROWS = WG / TPR;
  __shared__ float red0[WG / 64][1], red1[WG / 64][1], red2[WG / 64][2];
  __shared__ __attribute__((aligned(16))) float join[ROWS > 1 ? (ROWS - 1) * TPR * C * 8 : 4];
  const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const float inv = 1.0f / (float)p.K;
  float dw[C][8], db[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = db[c][e] = 0.f;

  struct Row { uint4 h[C], g[C], s[C]; };
  auto load = [&](int t) {
    Row v;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TPR + tid) * 8;
      v.h[c] = v.g[c] = v.s[c] = zero4();
      if (t < p.T && col < p.K) {
        v.h[c] = ldg16(p.h + (long)t * p.ldh + col);
        v.g[c] = ldg16(p.dy + (long)t * p.lddy + col);
        if (p.dsum) v.s[c] = ldg16(p.dsum + (long)t * p.ldds + col);
      }
    }
    return v;
  };
  Row next;
  if (AHEAD) next = load(blockIdx.x * ROWS + group);
  for (int t0 = blockIdx.x * ROWS; t0 < p.T; t0 += gridDim.x * ROWS) {
    const int t = t0 + group;
    Row now = AHEAD ? next : load(t);
    if (AHEAD && t0 + (int)gridDim.x * ROWS < p.T) next = load(t + gridDim.x * ROWS);
    // Each pass widens the row's bf16 anew (`opaque`): held in fp32 from pass to pass they would take
    // the registers that the sums and the next row's loads need.
    float mean = 0.f;
    if (!RMS) {
      float s[1] = {0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float h[8];
        widen(now.h[c], h);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += h[e];
      }
      row_sum<WAVES, 1>(s, red0);
      mean = s[0] * inv;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float h[8];
      opaque(now.h[c]);
      widen(now.h[c], h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = h[e] - mean;
        q[0] += (c * TPR + tid) * 8 < p.K ? d * d : 0.f;
      }
    }
    row_sum<WAVES, 1>(q, red1);
    const float r = 1.0f / sqrtf(q[0] * inv + p.eps);
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TPR + tid) * 8;
      opaque(now.h[c]);
      if (t >= p.T || col >= p.K) continue;
      float h[8], g[8], w[8];
      widen(now.h[c], h);
      widen(now.g[c], g);
      if (p.weight) ld8(p.weight + col, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (h[e] - mean) * r;
        dw[c][e] += g[e] * xh;
        db[c][e] += g[e];
        const float gw = p.weight ? g[e] * w[e] : g[e];
        m[0] += gw;
        m[1] += gw * xh;
      }
    }
    row_sum<WAVES, 2>(m, red2);
    const float m0 = RMS ? 0.f : m[0] * inv, m1 = m[1] * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TPR + tid) * 8;
      opaque(now.h[c]);
      opaque(now.g[c]);
      if (t >= p.T || col >= p.K) continue;
      float h[8], g[8], w[8], s[8];
      widen(now.h[c], h);
      widen(now.g[c], g);
      widen(now.s[c], s);
      if (p.weight) ld8(p.weight + col, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (h[e] - mean) * r, gw = p.weight ? g[e] * w[e] : g[e];
        g[e] = r * (gw - m0 - xh * m1) + s[e];
      }
      *reinterpret_cast<uint4*>(p.dx + (long)t * p.lddx + col) = narrow(g);
    }
  }
  // the workgroup's rows joined in LDS in order, into one row of partial sums
  const int n = (p.dweight ? 1 : 0) + (p.dbias ? 1 : 0);
  float* out = p.part + (long)blockIdx.x * n * p.K;
  auto write = [&](float (&a)[C][8]) {
    if (ROWS > 1) {
      __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float* at = join + ((group - 1) * C + c) * TPR * 8 + tid * 4;
          *reinterpret_cast<float4*>(at) = make_float4(a[c][0], a[c][1], a[c][2], a[c][3]);
          *reinterpret_cast<float4*>(at + TPR * 4) = make_float4(a[c][4], a[c][5], a[c][6], a[c][7]);
        }
      }
      __syncthreads();
    }
    if (group == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * TPR + tid) * 8;
#pragma unroll
        for (int i = 1; i < ROWS; ++i) {
          const float* at = join + ((i - 1) * C + c) * TPR * 8 + tid * 4;
          const float4 lo = *reinterpret_cast<const float4*>(at), hi = *reinterpret_cast<const float4*>(at + TPR * 4);
          a[c][0] += lo.x; a[c][1] += lo.y; a[c][2] += lo.z; a[c][3] += lo.w;
          a[c][4] += hi.x; a[c][5] += hi.y; a[c][6] += hi.z; a[c][7] += hi.w;
        }
        if (col < p.K) {
          *reinterpret_cast<float4*>(out + col) = make_float4(a[c][0], a[c][1], a[c][2], a[c][3]);
          *reinterpret_cast<float4*>(out + col + 4) = make_float4(a[c][4], a[c][5], a[c][6], a[c][7]);
        }
      }
    }
    out += p.K;
  };
  if (p.dweight) write(dw);
  if (p.dbias) write(db);
}

// Sums of the partial rows' columns, 64 columns a workgroup: 16 lanes of float4 by 64 rows, then a
// fixed order.
__global__ __launch_bounds__(1024) void k_norm_join(const float* __restrict__ part, int n_wg, int K, int n, float* first, float* second) {
  __shared__ float4 red[64][16];
  const int c4 = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const long all = (long)n * K, col = (long)blockIdx.x * 64 + 4 * c4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < all) {
#pragma unroll 4
    for (int r = rg; r < n_wg; r += 64) {
      const float4 u = *reinterpret_cast<const float4*>(part + r * all + col);
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
  }
  red[rg][c4] = v;
  __syncthreads();
  if (rg || col >= all) return;
#pragma unroll 8
  for (int w = 1; w < 64; ++w) {
    const float4 u = red[w][c4];
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  float* to = col < K ? first + col : second + (col - K);
  *reinterpret_cast<float4*>(to) = v;
}

template <int TPR, int C, int WG>
hipError_t launch_fwd(const NormParams& p, bool rms, hipStream_t s) {
  const dim3 grid((unsigned)((p.T + WG / TPR - 1) / (WG / TPR)));
  if (rms) hipLaunchKernelGGL((k_norm<TPR, C, WG, true>), grid, dim3(WG), 0, s, p);
  else hipLaunchKernelGGL((k_norm<TPR, C, WG, false>), grid, dim3(WG), 0, s, p);
  return hipGetLastError();
}

template <int TPR, int C, int WG, bool AHEAD>
hipError_t launch_bwd(NormBwdParams p, bool rms, hipStream_t s) {
  constexpr int ROWS = WG / TPR;
  p.n_wg = std::min(NORM_BWD_WGS, (p.T + ROWS - 1) / ROWS);
  if (p.T > 0) {
    if (rms) hipLaunchKernelGGL((k_norm_bwd<TPR, C, WG, AHEAD, true>), dim3(p.n_wg), dim3(WG), 0, s, p);
    else hipLaunchKernelGGL((k_norm_bwd<TPR, C, WG, AHEAD, false>), dim3(p.n_wg), dim3(WG), 0, s, p);
  }
  const int n = (p.dweight ? 1 : 0) + (p.dbias ? 1 : 0);
  if (n) {
    float *a = p.dweight ? p.dweight : p.dbias, *b = p.dbias;
    hipLaunchKernelGGL(k_norm_join, dim3((unsigned)(((long)n * p.K + 63) / 64)), dim3(1024), 0, s, p.part, p.n_wg, p.K, n, a, b);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormParams& p, bool rms, hipStream_t s) {
  if (p.K <= 2048) return launch_fwd<256, 1, 256>(p, rms, s);
  if (p.K <= 4096) return launch_fwd<256, 2, 256>(p, rms, s);
  if (p.K <= 8192) return launch_fwd<256, 4, 256>(p, rms, s);
  return launch_fwd<1024, 2, 1024>(p, rms, s);
}

hipError_t launch_norm_bwd(const NormBwdParams& p, bool rms, hipStream_t s) {
  if (p.K <= 512) return launch_bwd<64, 1, 1024, true>(p, rms, s);
  if (p.K <= 2048) return launch_bwd<256, 1, 1024, true>(p, rms, s);
  if (p.K <= 4096) return launch_bwd<256, 2, 512, true>(p, rms, s);
  if (p.K <= 8192) return launch_bwd<512, 2, 512, true>(p, rms, s);
  return launch_bwd<512, 4, 512, false>(p, rms, s);
}

}  // namespace lora
