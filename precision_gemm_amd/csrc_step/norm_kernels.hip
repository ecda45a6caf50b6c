// Layer norm and RMS norm of rows of hidden states, forward (with the residual's addition) and
// backward.
//
// Mathematics, for one row h of K values (mu = 0 for the RMS norm):
//   mu = mean(h),  r = 1 / sqrt(mean((h - mu)^2) + eps),  xh = (h - mu) r,  y = xh w + b
// and backwards, with g = dy w:
//   dh = r (g - mean(g) - xh mean(g xh))   (without mean(g) for the RMS norm)
//   dw = sum over the rows of dy xh,  db = sum of dy.
//
// Bound by HBM; a row is read once and held in registers, so the squares are summed about the mean (and
// the backward takes the statistics anew, without reading anything for it).
#include <algorithm>

#include "step_kernels.hpp"
#include "../csrc/device_common.hpp"
#include "../csrc_attn/row_buffer.hpp"

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

// s plus the sum of eight bf16: two products by 1 an instruction, exact, added in fp32.
__device__ __forceinline__ float sum8(const uint4& v, float s) {
#if defined(__HIP_DEVICE_COMPILE__)
  const bf16x2 one = __builtin_bit_cast(bf16x2, 0x3f803f80u);
  s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v.x), one, s, false);
  s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v.y), one, s, false);
  s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v.z), one, s, false);
  s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v.w), one, s, false);
#endif
  return s;
}

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

// TPR threads a row, C chunks of 8 values a thread, WG threads a workgroup.  4,096 rows of 4,096 values
// with a residual (134 MB): 21.5 us, 6.2 TB/s (a copy of as many bytes 26).  Loads under a condition
// instead of bounded buffers: 25.
template <int TPR, int C, int WG, bool RMS, bool RES>
__global__ __launch_bounds__(WG) void k_norm(NormParams p) {
  constexpr int WAVES = TPR / 64;
  __shared__ float red[2][WG / 64][1];
  const int tid = threadIdx.x % TPR;
  const int t = blockIdx.x * (WG / TPR) + __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);
  const bool row = t < p.T;
  const RowBuffer rx(p.x, p.ldx, t, p.K, row), ry(p.y, p.ldy, t, p.K, row);
  const RowBuffer rr(p.residual, p.ldr, t, p.K, RES && row), rs(p.sum, p.lds, t, p.K, RES && row);
  uint4 x[C], res[C];
#pragma unroll
  for (int c = 0; c < C; ++c) x[c] = rx.load((c * TPR + tid) * 8);
  if (RES) {
#pragma unroll
    for (int c = 0; c < C; ++c) res[c] = rr.load((c * TPR + tid) * 8);
  }
  float h[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    widen(x[c], h[c]);
    if (RES) {
      float r[8];
      widen(res[c], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] += h[c][e];
      const uint4 a = narrow(r);  // the stream's own rounding: the statistics are those of what is stored
      rs.store((c * TPR + tid) * 8, a);
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
  for (int c = 0; c < C; ++c) {
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[c][e] -= mean;
      part += h[c][e] * h[c][e];
    }
    q[0] += (c * TPR + tid) * 8 < p.K ? part : 0.f;
  }
  row_sum<WAVES, 1>(q, red[1]);
  const float r = 1.0f / sqrtf(q[0] / (float)p.K + p.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TPR + tid) * 8;
    float w[8], b[8];
    if (p.weight && col < p.K) ld8(p.weight + col, w);
    if (p.bias && col < p.K) ld8(p.bias + col, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = h[c][e] * r;
      if (p.weight) v *= w[e];
      if (p.bias) v += b[e];
      h[c][e] = v;
    }
    ry.store(col, narrow(h[c]));
  }
}

// Backward.  A workgroup takes rows blockIdx.x * (WG / TPR) + ... in strides of the grid, the loads of
// the next AHEAD of them in flight; a thread meets the same columns in every row, so it keeps their
// weights, and their sums for the weights' gradients, in registers.  One workgroup a CU (256 in all), for
// each leaves a row of partial sums (512: 20 % longer).  Sums meet a wave's lanes by DPP and its
// workgroup's waves through LDS, three times a row (twice for the RMS norm).  With the dot product taken
// beside the squares, about h - mu and scaled afterwards, it is once less: 2 to 4 % faster up to 2,048
// columns, 2 to 12 % slower from 8,192 on, where the registers are short.  4,096 rows of 4,096 values, with
// the residual stream's gradient (134 MB): 26.6 us, 5.0 TB/s, and k_norm_join.  Loads under a condition
// (which wait for the next row's): 36.
template <int TPR, int C, int WG, int AHEAD, bool RMS, bool DSUM>
__global__ __launch_bounds__(WG) void k_norm_bwd(NormBwdParams p) {
  constexpr int WAVES = TPR / 64, ROWS = WG / TPR;
  __shared__ float red0[WG / 64][1], red1[WG / 64][1], red2[WG / 64][RMS ? 1 : 2];
  __shared__ __attribute__((aligned(16))) float join[ROWS > 1 ? (ROWS - 1) * TPR * C * 8 : 4];
  const int tid = threadIdx.x % TPR, group = __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);
  const float inv = 1.0f / (float)p.K;
  float dw[C][8], db[C][8], w[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[c][e] = db[c][e] = 0.f;
      w[c][e] = 1.f;
    }
    if (p.weight && (c * TPR + tid) * 8 < p.K) ld8(p.weight + (c * TPR + tid) * 8, w[c]);
  }

  // four chunks a thread leave no registers for the residual stream's gradient ahead of its row
  constexpr bool SUM_AHEAD = DSUM && C * WG <= 1024;
  struct Row { uint4 h[C], g[C], s[C]; };
  auto load_sum = [&](int t, Row& v) {
    const RowBuffer rs(p.dsum, p.ldds, t, p.K, t < p.T);
#pragma unroll
    for (int c = 0; c < C; ++c) v.s[c] = rs.load((c * TPR + tid) * 8);
  };
  auto load = [&](int t) {
    const RowBuffer rh(p.h, p.ldh, t, p.K, t < p.T), rg(p.dy, p.lddy, t, p.K, t < p.T);
    Row v;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TPR + tid) * 8;
      v.h[c] = rh.load(col);
      v.g[c] = rg.load(col);
    }
    if (SUM_AHEAD) load_sum(t, v);
    return v;
  };
  auto row = [&](int t, const Row& now) {
    float h[C][8], g[C][8];  // h, then xh; dy, then g
#pragma unroll
    for (int c = 0; c < C; ++c) widen(now.h[c], h[c]);
    float mean = 0.f;
    if (!RMS) {
      float s[1] = {0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) s[0] = sum8(now.h[c], s[0]);
      row_sum<WAVES, 1>(s, red0);
      mean = s[0] * inv;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float part = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!RMS) h[c][e] -= mean;
        part += h[c][e] * h[c][e];
      }
      q[0] += (c * TPR + tid) * 8 < p.K ? part : 0.f;
    }
    row_sum<WAVES, 1>(q, red1);
    const float r = 1.0f / sqrtf(q[0] * inv + p.eps);
    float m[RMS ? 1 : 2] = {};  // g xh, and g
    if (t < p.T) {  // a row behind the last is all zeros, whose r may be infinite
#pragma unroll
      for (int c = 0; c < C; ++c) {
        widen(now.g[c], g[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[c][e] *= r;
          dw[c][e] += g[c][e] * h[c][e];
          db[c][e] += g[c][e];
          g[c][e] *= w[c][e];
          m[0] += g[c][e] * h[c][e];
          if (!RMS) m[RMS ? 0 : 1] += g[c][e];
        }
      }
    }
    row_sum<WAVES, RMS ? 1 : 2>(m, red2);
    const float m0 = RMS ? 0.f : m[RMS ? 0 : 1] * inv, m1 = m[0] * inv;
    const RowBuffer rx(p.dx, p.lddx, t, p.K, t < p.T);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float s[8];
      if (DSUM) widen(now.s[c], s);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = RMS ? g[c][e] - h[c][e] * m1 : g[c][e] - m0 - h[c][e] * m1;
        g[c][e] = DSUM ? r * v + s[e] : r * v;
      }
      rx.store((c * TPR + tid) * 8, narrow(g[c]));
    }
  };
  const int stride = gridDim.x * ROWS;
  Row ahead[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) ahead[i] = load((blockIdx.x + i * gridDim.x) * ROWS + group);
  // whole rounds of AHEAD rows: those behind the last are buffers of no bytes
  for (int t = blockIdx.x * ROWS + group; t < p.T + group; t += AHEAD * stride) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      Row now = ahead[i];
      if (DSUM && !SUM_AHEAD) load_sum(t + i * stride, now);
      ahead[i] = load(t + (i + AHEAD) * stride);
      row(t + i * stride, now);
    }
  }
  // the workgroup's rows joined in LDS in order, into one row of partial sums, or the result
  const int n = (p.dweight ? 1 : 0) + (p.dbias ? 1 : 0);
  float* row_out = p.part + (long)blockIdx.x * n * p.K;
  auto write = [&](float (&a)[C][8], float* result) {
    float* out = p.n_wg == 1 ? result : row_out;
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
    row_out += p.K;
  };
  if (p.dweight) write(dw, p.dweight);
  if (p.dbias) write(db, p.dbias);
}

// Sums of the partial rows' columns, 64 columns a workgroup: 16 lanes of float4 by 64 rows, then a
// fixed order.  256 rows of 8,192 (8.4 MB): 4.6 us, a launch and four rounds of loads.
__global__ __launch_bounds__(1024) void k_norm_join(const float* __restrict__ part, int n_wg, int K, int n, float* first, float* second) {
  __shared__ float4 red[16][16];
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
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) {
    v.x += __shfl_xor(v.x, d); v.y += __shfl_xor(v.y, d); v.z += __shfl_xor(v.z, d); v.w += __shfl_xor(v.w, d);
  }
  if ((threadIdx.x & 63) < 16) red[threadIdx.x >> 6][c4] = v;
  __syncthreads();
  if (rg || col >= all) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) {
    const float4 u = red[w][c4];
    v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
  }
  float* to = col < K ? first + col : second + (col - K);
  *reinterpret_cast<float4*>(to) = v;
}

template <int TPR, int C, int WG>
hipError_t launch_fwd(const NormParams& p, bool rms, hipStream_t s) {
  const dim3 grid((unsigned)((p.T + WG / TPR - 1) / (WG / TPR)));
  if (rms && p.residual) hipLaunchKernelGGL((k_norm<TPR, C, WG, true, true>), grid, dim3(WG), 0, s, p);
  else if (rms) hipLaunchKernelGGL((k_norm<TPR, C, WG, true, false>), grid, dim3(WG), 0, s, p);
  else if (p.residual) hipLaunchKernelGGL((k_norm<TPR, C, WG, false, true>), grid, dim3(WG), 0, s, p);
  else hipLaunchKernelGGL((k_norm<TPR, C, WG, false, false>), grid, dim3(WG), 0, s, p);
  return hipGetLastError();
}

template <int TPR, int C, int WG, int AHEAD>
hipError_t launch_bwd(NormBwdParams p, bool rms, hipStream_t s) {
  constexpr int ROWS = WG / TPR;
  p.n_wg = std::min(NORM_BWD_WGS, (p.T + ROWS - 1) / ROWS);
  if (p.T > 0) {
    const dim3 grid(p.n_wg), wg(WG);
    if (rms && p.dsum) hipLaunchKernelGGL((k_norm_bwd<TPR, C, WG, AHEAD, true, true>), grid, wg, 0, s, p);
    else if (rms) hipLaunchKernelGGL((k_norm_bwd<TPR, C, WG, AHEAD, true, false>), grid, wg, 0, s, p);
    else if (p.dsum) hipLaunchKernelGGL((k_norm_bwd<TPR, C, WG, AHEAD, false, true>), grid, wg, 0, s, p);
    else hipLaunchKernelGGL((k_norm_bwd<TPR, C, WG, AHEAD, false, false>), grid, wg, 0, s, p);
  }
  const int n = (p.dweight ? 1 : 0) + (p.dbias ? 1 : 0);
  if (n && p.n_wg != 1) {  // one workgroup's sums are the result
    float *a = p.dweight ? p.dweight : p.dbias, *b = p.dbias;
    hipLaunchKernelGGL(k_norm_join, dim3((unsigned)(((long)n * p.K + 63) / 64)), dim3(1024), 0, s, p.part, p.n_wg, p.K, n, a, b);
  }
  return hipGetLastError();
}

}  // namespace

// Threads and chunks by the row's width.  8,192 rows of 512: one wave a row 7.3 us, a workgroup of 256
// threads 12.6; 4,096 rows of 4,096 (256 threads, 2 chunks 21.2 us; 512 x 1 21.4, 128 x 4 22.0, 64 x 8 23.6)
// and of 8,192 (512 x 2 42.5; 256 x 4 43.5, 1024 x 1 44.3, 128 x 8 46.0); 2,048 of 16,384 (1024 x 2 47.6;
// 512 x 4 49.6, 256 x 8 50.0).
hipError_t launch_norm(const NormParams& p, bool rms, hipStream_t s) {
  if (p.K <= 512) return launch_fwd<64, 1, 64>(p, rms, s);
  if (p.K <= 1024) return launch_fwd<128, 1, 128>(p, rms, s);
  if (p.K <= 2048) return launch_fwd<256, 1, 256>(p, rms, s);
  if (p.K <= 4096) return launch_fwd<256, 2, 256>(p, rms, s);
  if (p.K <= 8192) return launch_fwd<512, 2, 512>(p, rms, s);
  return launch_fwd<1024, 2, 1024>(p, rms, s);
}

// The same, and rows at a time of a workgroup (its threads by those of a row).  With k_norm_join: 8,192 rows
// of 512 in workgroups of 512 threads 11.3 us, of 1,024 11.8, of 256 12.4; of 2,048 (128 threads, 2 chunks,
// 4 rows 23.2; 256 x 1, 4 rows 24.0); 4,096 of 4,096 (256 x 2, 2 rows 30.2, two rows ahead 30.2; 512 x 1,
// 2 rows 31.1); 1,001 of 5,376 (384 x 2, 2 rows 13.1; 512 x 2 15.6); 4,096 of 8,192 (1024 x 1 49.7; 512 x 2
// 50.9); 2,048 of 16,384 (512 x 4 66; 1024 x 2 spills, 89), whose form also takes 8,200 columns and more
// (4,096 rows of 8,200 73.9 us, of 10,240 77.1, of 12,288 84.5; 768 x 2 73.9, 77.1 and 85.7).  Without the
// weights' gradients the sums are kept all the same, and no k_norm_join follows: 4,096 of 4,096 25.8 us
// where both take 31.8 and one 30.1.
hipError_t launch_norm_bwd(const NormBwdParams& p, bool rms, hipStream_t s) {
  if (p.K <= 512) return launch_bwd<64, 1, 512, 1>(p, rms, s);
  if (p.K <= 1024) return launch_bwd<128, 1, 512, 1>(p, rms, s);
  if (p.K <= 2048) return launch_bwd<128, 2, 512, 1>(p, rms, s);
  if (p.K <= 4096) return launch_bwd<256, 2, 512, 1>(p, rms, s);
  if (p.K <= 6144) return launch_bwd<384, 2, 768, 1>(p, rms, s);
  if (p.K <= 8192) return launch_bwd<1024, 1, 1024, 1>(p, rms, s);
  return launch_bwd<512, 4, 512, 1>(p, rms, s);
}

}  // namespace lora
