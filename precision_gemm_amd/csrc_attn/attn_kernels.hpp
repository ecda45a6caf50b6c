// Internal interface between the host layer of the attention block (attn_api.cpp) and its
// gfx950 kernels (rope_kernels.hip, tree_attention.hip).  Not part of the public header.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/lora_lowp.h"

namespace lora {

// Positions of several axes: pair i of a head turns by the position on axis (pair[i / 32] >> 2 (i % 32)) & 3.
struct AxisMap {
  uint64_t pair[4];
  uint64_t quad;           // the same for each four pairs, where all quads have one axis
  int n;                   // axes; 0: one position a token
  int quads;               // each quad of pairs has one axis
};

// Head norm and rotation, forward (k_out) and into the paged cache (k_cache).
struct RopeParams {
  const uint16_t* qkv;     // bf16 [T][ld]: n_q, n_kv, n_kv heads of D
  long ld;
  const int* positions;    // [T], or [axes.n][T]
  int T, n_q, n_kv;
  const float* cos_sin;    // [max_pos][rot]: rot / 2 cosines, then the sines
  int max_pos, rot, interleaved;
  const float *q_weight, *k_weight;  // both or neither
  float eps;
  uint16_t* q_out;
  long ldq;
  uint16_t* k_out;         // forward only
  long ldk;
  const int* slots;        // append only
  void *k_cache, *v_cache; // [n_pages][n_kv][page][D]
  const float *k_scale, *v_scale;
  int page_log2;
  long n_slots;
  int* status;
  int rounds_q, rounds_k;  // waves over a token's query heads, key (and value) heads
  AxisMap axes;
};

struct RopeBwdParams {
  const uint16_t* qkv;
  long ld;
  const int* positions;
  int T, n_q, n_kv;
  const float* cos_sin;
  int max_pos, rot, interleaved;
  const float *q_weight, *k_weight;
  float eps;
  const uint16_t *dq, *dk, *dv;      // dense rows; dv may be null
  uint16_t* dqkv;
  long ldd;
  float* part;                       // [n_wg][D]
  float *dqw, *dkw;
  int* status;
  int rounds_q, rounds_k;            // rounds of a wave over a token's query heads, key heads
  int q_wg, n_wg;                    // workgroups of the query heads, of all
  AxisMap axes;
};

constexpr int ROPE_BWD_WGS = 768;    // most workgroups of the backward (three a CU) and rows of its partial sums

hipError_t launch_norm_rope(const RopeParams& p, int D, hipStream_t s);
hipError_t launch_rope_append(const RopeParams& p, int D, bool fp8, hipStream_t s);
hipError_t launch_norm_rope_bwd(const RopeBwdParams& p, int D, hipStream_t s);

// Attention over the paged cache.
struct TreeAttnParams {
  const uint16_t* q;       // bf16 [T][ldq]
  long ldq;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;    // 8-bit cache only
  const int* page_table;   // [B][max_pages]
  int max_pages, n_pages, page_log2;
  const int *kv_len, *q_indptr;
  int B, T, max_q, n_q, n_kv, group;
  const uint64_t* mask;    // [T][words], or null (causal)
  int words;
  float scale_log2;        // the softmax scale times log2(e)
  uint16_t* out;           // bf16 [T][n_q][D]
  float* lse;              // [T][n_q], may be null
  int* desc;               // [n_wg][ATTN_DESC]: a unit that this workgroup began and others end
  float* part_ml;          // [2 n_wg][rows][2]
  float* part_o;           // [2 n_wg][rows][D]
  int n_wg;
  int counted;             // a row block counts the steps that its tokens see, not all
  int* status;
};

constexpr int ATTN_MAX_B = 4096;     // sequences of one call (their prefix sums live in LDS)
constexpr int ATTN_DESC = 8;         // words of a cut unit's description
constexpr int ATTN_GROUP = 32;       // keys of one MFMA group
constexpr int ATTN_KEYS = 128;       // keys of a step: a group for each of four waves, or a round of four groups

// How a call's rows (drafted tokens times query heads of a kv head) are taken: by waves that
// split a step's keys, or (`shared`) that share them; row tiles of 16 a wave holds, rows of a
// workgroup, workgroups; whether in-order row blocks are `counted` by what they see.  `heads`: kv
// heads of all the call's sequences.
struct TreeAttnPlan { bool shared, counted; int row_tiles, block_rows, n_wg; size_t desc_bytes, ml_bytes, o_bytes; };
TreeAttnPlan tree_attn_plan(int D, int max_q, int group, bool fp8, bool mask, long heads);
hipError_t launch_tree_attention(const TreeAttnParams& p, const TreeAttnPlan& pl, int D, bool fp8, hipStream_t s);
hipError_t launch_tree_mask(const int* parents, const int* q_indptr, int B, int T, int max_q, int words, uint64_t* mask,
                            int* status, hipStream_t s);

}  // namespace lora
