// Internal interface between the host layer of what stands around the low-precision layer in a
// step (step_api.cpp) and its gfx950 kernels (norm_kernels.hip, adamw_kernels.hip).  Not part of
// the public header.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/lora_lowp.h"

namespace lora {

// Norm of rows, forward.
struct NormParams {
  const uint16_t* x;         // bf16 [T][ldx]
  long ldx;
  const uint16_t* residual;  // bf16 [T][ldr], or null
  long ldr;
  int T, K;
  const float *weight, *bias;  // [K], or null
  float eps;
  uint16_t* y;
  long ldy;
  uint16_t* sum;             // bf16 [T][lds], with a residual
  long lds;
};

struct NormBwdParams {
  const uint16_t* dy;
  long lddy;
  const uint16_t* h;
  long ldh;
  const float* weight;
  const uint16_t* dsum;      // or null
  long ldds;
  int T, K;
  float eps;
  uint16_t* dx;
  long lddx;
  float *dweight, *dbias;    // [K], or null
  float* part;               // [n_wg][1 or 2][K]
  int n_wg;
};

constexpr int NORM_MAX_K = 16384;
constexpr int NORM_BWD_WGS = 256;  // most workgroups of the backward (one a CU) and rows of its partial sums

// An AdamW step over many tensors.
struct AdamWParams {
  const lora_adamw_tile* tiles;
  long n_tiles;
  const int* group_first;    // [n_groups + 1]: the groups' tiles
  int n_groups;
  const double* hyper;       // [n_groups][ADAMW_HYPER]
  const int* active;         // [n_groups], or null: all
  int* steps;
  float* norm;               // [n_groups], or null: no norms, no clipping
  int* status;
  double* part;              // [n_tiles]: sums of squares
  float* coef;               // [n_groups][ADAMW_COEF]
  int* arrived;              // [n_groups][ADAMW_LINE]: tiles of the group that are done; 0 between calls
};

constexpr int ADAMW_HYPER = 6;   // rate, beta1, beta2, eps, weight decay, largest norm
constexpr int ADAMW_COEF = 12;
constexpr int ADAMW_LINE = 32;   // words of a cache line: each group's arrivals on a line of their own
constexpr int ADAMW_TILE = 4096; // most values of a tile
constexpr int ADAMW_BLOCK = 64;  // values that share a scale of the 8-bit states

// Rows of A (columns of B) that a tile takes, for rank r: 4,096 values for ranks of 16, 32 and 64.  Small
// ranks write more padding than values, and tiles of 4,096 of them take longer than they save (rank 8,
// one adapter of 4096 x 4096: 512 rows 6.2 us, 256 rows 5.4).
inline __host__ __device__ int adamw_tile_span(int r) { return r <= 4 ? 512 : r <= 16 ? 256 : r <= 32 ? 128 : 64; }

hipError_t launch_adamw(const AdamWParams& p, int state_bits, hipStream_t s);

hipError_t launch_norm(const NormParams& p, bool rms, hipStream_t s);
hipError_t launch_norm_bwd(const NormBwdParams& p, bool rms, hipStream_t s);

}  // namespace lora
