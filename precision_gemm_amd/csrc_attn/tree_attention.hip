// Attention for a tree of drafted tokens over a paged cache.
//
//   S_rk = scale q_r . K_k,   O_r = sum_k exp(S_rk - m_r) V_k / l_r,   l_r = sum_k exp(S_rk - m_r)
//
// over the keys k that row r sees: every cached key before the drafted ones, and of those
// the ones its mask names (without a mask: those up to itself).  One pass over the keys with
// a running maximum m and sum l; the running reference is only moved when a score exceeds it
// by 2^8 (the sums are in 32 bits, so exp(S - m) <= 2^8 costs nothing), which takes the
// rescaling and the maximum's exchange between lanes out of almost every step.
//
// Split: the keys of all (sequence, kv head, row block) units form one line of steps of 128
// keys; every workgroup takes an equal stretch of it, whatever the sequences' lengths, and
// finds its place from a prefix sum over the sequences that it computes itself, so the host
// needs no lengths.  A unit cut between workgroups leaves its pieces (m, l, unnormalised O in
// 32 bits) in the workspace; k_tree_combine joins them in order.
//
// Layout: a wave takes 32 keys of a step and all rows of its unit (the query heads that share
// the kv head, times the drafted tokens).  It forms S^T = K Q^T (16x16x32 bf16 MFMA), whose
// result layout, with key rows dealt to the two 16-key tiles in fours, is the operand layout
// of O^T = V^T P^T as it stands: probabilities never leave their lane.  K rows are MFMA
// operands as loaded; V rows are transposed in registers, a lane's 8 keys x CH values by byte
// permutes.  Nothing goes through LDS until the four waves' results are joined at the end of
// a unit, so every cached byte is loaded once per row block, straight into registers, and the
// loads of the next step's K are issued as soon as this step's are used, then V's likewise.
#include <type_traits>

#include "attn_kernels.hpp"
#include "../csrc/device_common.hpp"

namespace lora {
namespace {

constexpr int ST_PAGE = 4, ST_LENGTH = 8, ST_PARENT = 16;  // LORA_ATTN_BAD_PAGE, _BAD_LENGTH, _BAD_PARENT
constexpr float NEG_INF = -__builtin_inff();
constexpr float SLACK = 8.0f;  // log2 units a score may exceed the running reference by

template <int D, bool FP8>
struct Geo {
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int ROWB = D * ESZ;                  // bytes of a cached row
  static constexpr int KS = D / 32;                     // MFMA steps over the head
  static constexpr int KL = ROWB / 64;                  // 16-byte K loads of a lane for 16 keys
  static constexpr int VB = ROWB / 16 > 16 ? 16 : ROWB / 16;  // bytes of a lane's V load
  static constexpr int VW = VB / 4;
  static constexpr int CH = VB / ESZ;                   // consecutive values of a lane's V load
  static constexpr int NCH = D / (16 * CH);             // V loads of a lane for one key
};

// place in the head of the 8 values of MFMA step s that lane group g holds
template <bool FP8>
__device__ __forceinline__ int q_place(int s, int g) {
  return FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
}

// A table entry at an address that is the same for the whole wave, through the scalar cache
// (the call's index tables are not written while it runs).
__device__ __forceinline__ int ld_table(const int* p) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(4))) const int c_int;
  return *(c_int*)(reinterpret_cast<uintptr_t>(p));
#else
  return *p;  // host pass only; never executed
#endif
}

template <int BYTES>
__device__ __forceinline__ void ldg_words(const char* p, uint32_t* w) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (BYTES == 16) {
    const uint4 v = ldg16(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    typedef __attribute__((address_space(1))) const uint2 g_uint2;
    const uint2 v = *(g_uint2*)(reinterpret_cast<uintptr_t>(p));
    w[0] = v.x; w[1] = v.y;
  } else {
    typedef __attribute__((address_space(1))) const uint32_t g_u32;
    w[0] = *(g_u32*)(reinterpret_cast<uintptr_t>(p));
  }
#endif
}

// Which of the 8 keys at draft places d0 .. d0 + 7 (negative: before the drafted tokens) the
// drafted token j of n sees.  mrow: its mask words, or null for the causal rule.
__device__ __forceinline__ uint32_t visible8(const uint64_t* mrow, int words, int j, int d0, int n) {
  if (d0 <= -8) return 0xffu;
  if (d0 >= n) return 0u;
  uint32_t bits;
  if (!mrow) {
    const int c = j - d0 + 1;
    bits = c >= 8 ? 0xffu : c <= 0 ? 0u : (1u << c) - 1u;
  } else if (d0 < 0) {
    bits = ((uint32_t)mrow[0] << -d0) | ((1u << -d0) - 1u);
  } else {
    const int w = d0 >> 6, o = d0 & 63;
    uint64_t v = mrow[w] >> o;
    if (o > 56 && w + 1 < words) v |= mrow[w + 1] << (64 - o);
    bits = (uint32_t)v;
  }
  const int keep = n - d0;
  if (keep < 8) bits &= (1u << keep) - 1u;
  return bits & 0xffu;
}

// One sequence: its queries and keys, and how many units and steps they make.
struct Seq { int q0, n, kv, steps, blocks; bool bad; };
__device__ __forceinline__ Seq make_seq(const TreeAttnParams& p, int q0, int q1, int kv, int block_rows) {
  Seq s;
  s.q0 = q0;
  s.kv = kv;
  s.bad = false;
  s.n = q1 - q0;
  if (q0 < 0 || q1 > p.T || s.n < 0 || s.n > p.max_q) { s.n = 0; s.bad = true; }
  if (kv < s.n || (long)kv > ((long)p.max_pages << p.page_log2)) { s.kv = 0; s.bad = true; }
  s.steps = max(1, (s.kv + ATTN_KEYS - 1) / ATTN_KEYS);
  s.blocks = (s.n * p.group + block_rows - 1) / block_rows;
  return s;
}

// Prefix sum of the sequences' work in LDS: cum[b] steps before sequence b, cum[B] in all.
__device__ __forceinline__ void work_prefix(const TreeAttnParams& p, int block_rows, int* cum, int* wave_sum) {
  const int tid = threadIdx.x, lane = tid & 63, per = (p.B + 255) / 256;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < p.B) {
      const Seq s = make_seq(p, p.q_indptr[b], p.q_indptr[b + 1], p.kv_len[b], block_rows);
      if (s.bad && blockIdx.x == 0 && p.status) or_agent(p.status, ST_LENGTH);
      mine += p.n_kv * s.blocks * s.steps;
      cum[b + 1] = mine;
    }
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wave_sum[tid >> 6] = incl;
  __syncthreads();
  int before = incl - mine;
  for (int w = 0; w < (tid >> 6); ++w) before += wave_sum[w];
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < p.B) cum[b + 1] += before;
  }
  if (tid == 0) cum[0] = 0;
  __syncthreads();
}

// Write one finished row: four values of out and, once, lse.  No key seen: L is 0, else it is
// at least 1 (the score that set m), or not a number.
template <int D>
__device__ __forceinline__ void put_row(const TreeAttnParams& p, int q0, int h, int r, int c4, const float4& a, float M, float L,
                                        float vs) {
  const float inv = L == 0.f ? 0.f : vs / L;
  const int j = r / p.group;
  const long at = (long)(q0 + j) * p.n_q + h * p.group + (r - j * p.group);
  *reinterpret_cast<uint2*>(p.out + at * D + 4 * c4) = make_uint2(bf16x2_rne(a.x * inv, a.y * inv), bf16x2_rne(a.z * inv, a.w * inv));
  if (c4 == 0 && p.lse) p.lse[at] = L == 0.f ? NEG_INF : (M + __builtin_amdgcn_logf(L)) * 0.69314718055994531f;
}

template <int D, int RT, bool FP8, int OCC>
__global__ __launch_bounds__(256, OCC) void k_tree_attention(TreeAttnParams p) {
  using G = Geo<D, FP8>;
  constexpr int NT = D / 16;       // 16-row tiles of O^T
  constexpr int OS = D + 4;        // row stride of the joining buffer (floats)
  __shared__ __attribute__((aligned(16))) float so[4 * 16 * OS];
  __shared__ float sml[4][RT * 16][2];
  __shared__ int wave_sum[4], first_seq;
  // heads of 256: the queries are kept in LDS as operands, their registers hold keys and values
  constexpr bool Q_LDS = D == 256;
  static_assert(!Q_LDS || RT == 1, "one row tile in LDS");
  __shared__ uint4 sq_ops[Q_LDS ? G::KS : 1][64];
  extern __shared__ int cum[];     // [B + 1]

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // workgroups go to the eight XCDs in turn: give each XCD one stretch of the line, so that
  // neighbours, which read the same queries and (row blocks of a unit) the same keys, share an L2
  const int wg = (blockIdx.x & 7) * (p.n_wg >> 3) + (blockIdx.x >> 3);

  work_prefix(p, RT * 16, cum, wave_sum);
  const int total = cum[p.B];
  const int per = (total + p.n_wg - 1) / p.n_wg;
  int cur = wg * per;
  const int end = min(total, cur + per);
  if (tid == 0) p.desc[4 * wg] = 0;
  if (cur >= end) return;

  for (int c = tid; c < p.B; c += 256)
    if (cum[c] <= cur && cur < cum[c + 1]) first_seq = c;
  __syncthreads();
  int b = __builtin_amdgcn_readfirstlane(first_seq);
  cur = __builtin_amdgcn_readfirstlane(cur);

  const int page = 1 << p.page_log2;
  const int koff = (8 * ((i >> 2) & 1) + (i & 3)) * G::ROWB + 16 * g;
  const int voff = 8 * (g & 1) * G::ROWB + i * G::VB;

  while (cur < end) {
    while (cum[b + 1] <= cur) ++b;  // skips sequences without queries
    b = __builtin_amdgcn_readfirstlane(b);
    const Seq sq = make_seq(p, ld_table(p.q_indptr + b), ld_table(p.q_indptr + b + 1), ld_table(p.kv_len + b), RT * 16);
    const int local = cur - __builtin_amdgcn_readfirstlane(cum[b]);
    const int unit = local / sq.steps, t0 = local - unit * sq.steps;
    const int t1 = min(sq.steps, t0 + end - cur);
    const int h = unit / sq.blocks, rb = unit - h * sq.blocks;
    const int rows = sq.n * p.group, prefix = sq.kv - sq.n, kv = sq.kv;
    const int* table = p.page_table + (long)b * p.max_pages;

    // queries: column i of row tile rt is row (rb RT + rt) 16 + i = (token j, head of the group)
    uint4 q[RT][Q_LDS ? 1 : G::KS];
    int jrow[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = (rb * RT + rt) * 16 + i;
      const int j = r / p.group;
      jrow[rt] = min(j, sq.n - 1);
      const uint16_t* src = p.q + (long)(sq.q0 + jrow[rt]) * p.ldq + (long)(h * p.group + (r - j * p.group)) * D;
      if constexpr (Q_LDS) {
        for (int s = wave; s < G::KS; s += 4) sq_ops[s][lane] = r < rows ? ldg16(src + q_place<FP8>(s, g)) : zero4();
      } else {
#pragma unroll
        for (int s = 0; s < G::KS; ++s) q[rt][s] = r < rows ? ldg16(src + q_place<FP8>(s, g)) : zero4();
      }
    }
    if constexpr (Q_LDS) __syncthreads();
    const float sc = FP8 ? p.scale_log2 * p.k_scale[h] : p.scale_log2;

    v4f o[RT][NT];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = NEG_INF;
      l[rt] = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t) o[rt][t] = v4f{0.f, 0.f, 0.f, 0.f};
    }

    uint4 kr[2][G::KL];
    uint32_t vr[8][G::NCH * G::VW];
    // this wave's step: keys key0 .. key0 + 31 in two halves of 16, each within one page
    auto lookup = [&](int key0, int& p0, int& p1) {
      const int last = (kv - 1) >> p.page_log2;
      p0 = ld_table(table + min(key0 >> p.page_log2, last));
      p1 = ld_table(table + min((key0 + 16) >> p.page_log2, last));
    };
    auto row_base = [&](int id, int key) {  // byte offset of the half's first row
      const int ok = (unsigned)id < (unsigned)p.n_pages ? id : 0;
      return ((((long)ok * p.n_kv + h) << p.page_log2) + (key & (page - 1))) * G::ROWB;
    };
    auto load_k = [&](long b0, long b1) {
      const char* src = reinterpret_cast<const char*>(p.k_cache) + (i < 8 ? b0 : b1) + koff;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int c = 0; c < G::KL; ++c) kr[kt][c] = ldg16(src + kt * 4 * G::ROWB + 64 * c);
    };
    auto load_v = [&](long b0, long b1) {
      const char* src = reinterpret_cast<const char*>(p.v_cache) + (g < 2 ? b0 : b1) + voff;
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int c = 0; c < G::NCH; ++c) ldg_words<G::VB>(src + e * G::ROWB + c * 16 * G::VB, &vr[e][c * G::VW]);
    };

    constexpr int VE = G::NCH * G::CH / 2;  // words of a lane's V values of one key, in bf16
    auto widen_v = [](const uint32_t* in, uint32_t* out) {
      if constexpr (FP8) {
#pragma unroll
        for (int w = 0; w < G::NCH * G::VW; ++w) {
          const uint2 u = fp8x4_to_bf16(in[w]);
          out[2 * w] = u.x;
          out[2 * w + 1] = u.y;
        }
      } else {
#pragma unroll
        for (int w = 0; w < VE; ++w) out[w] = in[w];
      }
    };
    int key0 = t0 * ATTN_KEYS + wave * 32;
    int id0 = 0, id1 = 0, n0 = 0, n1 = 0;  // pages of this step and of the next one
    long b0 = 0, b1 = 0;
    if (key0 < kv) {
      lookup(key0, id0, id1);
      lookup(key0 + ATTN_KEYS, n0, n1);
      b0 = row_base(id0, key0);
      b1 = row_base(id1, key0 + 16);
      load_k(b0, b1);
      load_v(b0, b1);
    }
    // One step of this wave: SPECIAL where it reaches the drafted keys, the cache's end or a page
    // that does not exist.
    auto step = [&](auto special_t, bool more, long nb0, long nb1, bool bad0, bool bad1) {
      constexpr bool SPECIAL = decltype(special_t)::value;
      if constexpr (Q_LDS) asm volatile("" ::: "memory");  // re-read the queries, keep no copy in registers
      v4f s[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < G::KS; ++st) {
        uint4 qs = zero4();
        if constexpr (Q_LDS) qs = sq_ops[st][lane];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          uint4 a;
          if constexpr (FP8) {
            const uint4 w = kr[kt][st >> 1];
            const uint2 lo = fp8x4_to_bf16((st & 1) ? w.z : w.x), hi = fp8x4_to_bf16((st & 1) ? w.w : w.y);
            a = make_uint4(lo.x, lo.y, hi.x, hi.y);
          } else {
            a = kr[kt][st];
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) s[rt][kt] = mfma_bf16_16x16x32(a, Q_LDS ? qs : q[rt][Q_LDS ? 0 : st], s[rt][kt]);
        }
      }
      if (!SPECIAL && more) load_k(nb0, nb1);

      const int d0 = key0 + 8 * g - prefix;  // draft place of this lane's 8 keys
      const bool gone = g < 2 ? bad0 : bad1;
      uint4 pb[RT];
      uint32_t vis[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float x[8];  // scores of keys 8 g + e, in log2 units
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s[rt][e >> 2][e & 3] * sc;
        if constexpr (SPECIAL) {
          const uint64_t* mrow = p.mask ? p.mask + (long)(sq.q0 + jrow[rt]) * p.words : nullptr;
          vis[rt] = gone ? 0u : visible8(mrow, p.words, jrow[rt], d0, sq.n);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = (vis[rt] >> e) & 1u ? x[e] : NEG_INF;
        }
        float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        if (__any(mx > m[rt] + SLACK)) {
          mx = fmaxf(mx, __shfl_xor(mx, 16));
          mx = fmaxf(mx, __shfl_xor(mx, 32));
          // each row by its own scores alone: what a row gets does not depend on its neighbours
          const bool up = mx > m[rt] + SLACK;
          const float f = up ? __builtin_amdgcn_exp2f(m[rt] - mx) : 1.f;
          m[rt] = up ? mx : m[rt];
          l[rt] *= f;
#pragma unroll
          for (int tt = 0; tt < NT; ++tt) o[rt][tt] *= f;
        }
        const float ref = m[rt] == NEG_INF ? 0.f : m[rt];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = __builtin_amdgcn_exp2f(x[e] - ref);
          l[rt] += x[e];
        }
        // P enters the MFMA in bf16 (relative error 2^-8 an element at most, as the output's own
        // rounding); its sum l is taken before the rounding, in 32 bits
        pb[rt] = make_uint4(bf16x2_rne(x[0], x[1]), bf16x2_rne(x[2], x[3]), bf16x2_rne(x[4], x[5]), bf16x2_rne(x[6], x[7]));
      }

      // V: 8 keys x CH values a lane, widened to bf16
      uint32_t vb[8][VE];
#pragma unroll
      for (int e = 0; e < 8; ++e) widen_v(vr[e], vb[e]);
      uint32_t odd = 0;  // keys of this lane's group with a value that is not finite
      if constexpr (SPECIAL) {
        // Keys past the end, and of pages that do not exist, hold anything: their rows are
        // zeroed.  A drafted key that only some rows see must not reach the others through
        // 0 * NaN, so rows with values that are not finite are taken out of the product and
        // added apart, to the rows that see them.
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool none = gone || d0 + e >= sq.n;
          bool inf = false;
#pragma unroll
          for (int w = 0; w < VE; ++w) {
            vb[e][w] = none ? 0u : vb[e][w];
            inf |= ((vb[e][w] & 0x7f80u) == 0x7f80u) | ((vb[e][w] & 0x7f800000u) == 0x7f800000u);
          }
          const uint64_t any = __ballot(inf);
          if ((any >> (16 * g)) & 0xffffu) {
            odd |= 1u << e;
#pragma unroll
            for (int w = 0; w < VE; ++w) vb[e][w] = 0u;
          }
        }
      }
#pragma unroll
      for (int c = 0; c < G::NCH; ++c)
#pragma unroll
        for (int e = 0; e < G::CH; ++e) {
          const int w = c * (G::CH / 2) + (e >> 1);
          const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
          const uint4 a = make_uint4(__builtin_amdgcn_perm(vb[1][w], vb[0][w], sel), __builtin_amdgcn_perm(vb[3][w], vb[2][w], sel),
                                     __builtin_amdgcn_perm(vb[5][w], vb[4][w], sel), __builtin_amdgcn_perm(vb[7][w], vb[6][w], sel));
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) o[rt][c * G::CH + e] = mfma_bf16_16x16x32(a, pb[rt], o[rt][c * G::CH + e]);
        }
      if constexpr (SPECIAL) {
        for (int kk = 0; kk < 32; ++kk) {
          const int gk = kk >> 3, e = kk & 7;
          if (!((__builtin_amdgcn_readlane((int)odd, 16 * gk) >> e) & 1)) continue;
          // this key's row alone, as the operand whose only key it is
          const char* row = reinterpret_cast<const char*>(p.v_cache) + (gk < 2 ? b0 : b1) + (kk & 15) * G::ROWB + i * G::VB;
          uint32_t w1[G::NCH * G::VW], v1[VE];
#pragma unroll
          for (int c = 0; c < G::NCH; ++c) ldg_words<G::VB>(row + c * 16 * G::VB, &w1[c * G::VW]);
          widen_v(w1, v1);
          bool sees[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) sees[rt] = (__shfl((int)vis[rt], 16 * gk + i) >> e) & 1;
#pragma unroll
          for (int tt = 0; tt < NT; ++tt) {
            const uint32_t half = (v1[tt >> 1] >> (16 * (tt & 1))) & 0xffffu;
            const uint32_t val = g == gk ? half << (16 * (e & 1)) : 0u;
            const uint4 a = make_uint4((e >> 1) == 0 ? val : 0u, (e >> 1) == 1 ? val : 0u, (e >> 1) == 2 ? val : 0u, (e >> 1) == 3 ? val : 0u);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              const v4f add = mfma_bf16_16x16x32(a, pb[rt], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
              for (int r = 0; r < 4; ++r) o[rt][tt][r] += sees[rt] ? add[r] : 0.f;
            }
            __builtin_amdgcn_sched_barrier(0);  // one tile at a time: this path is rare, its registers are not
          }
        }
        if ((bad0 || bad1) && lane == 0 && p.status) or_agent(p.status, ST_PAGE);
        if (more) load_k(nb0, nb1);  // a unit's few last steps: its registers serve the above till here
      }
      if (more) load_v(nb0, nb1);
    };

    for (int t = t0; t < t1; ++t, key0 += ATTN_KEYS) {
      if (key0 >= kv) break;  // the last step's tail: nothing for this wave
      const int next = key0 + ATTN_KEYS;
      const bool more = t + 1 < t1 && next < kv;
      const long nb0 = row_base(n0, next), nb1 = row_base(n1, next + 16);
      int f0, f1;
      lookup(next + ATTN_KEYS, f0, f1);
      const bool bad0 = (unsigned)id0 >= (unsigned)p.n_pages, bad1 = (unsigned)id1 >= (unsigned)p.n_pages;
      if (key0 + 32 > prefix || bad0 || bad1)
        step(std::true_type{}, more, nb0, nb1, bad0, bad1);
      else
        step(std::false_type{}, more, nb0, nb1, false, false);
      id0 = n0; id1 = n1; n0 = f0; n1 = f1; b0 = nb0; b1 = nb1;
    }

    // join the four waves
    const bool whole = t0 == 0 && t1 == sq.steps;
    const int slot = 2 * wg + (t0 == 0 ? 1 : 0);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] += __shfl_xor(l[rt], 16);
      l[rt] += __shfl_xor(l[rt], 32);
      if (g == 0) {
        sml[wave][rt * 16 + i][0] = m[rt];
        sml[wave][rt * 16 + i][1] = l[rt];
      }
    }
    __syncthreads();
    const float vs = FP8 ? p.v_scale[h] : 1.f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if ((rb * RT + rt) * 16 < rows) {
        const int c = rt * 16 + i;
        const float mm = fmaxf(fmaxf(sml[0][c][0], sml[1][c][0]), fmaxf(sml[2][c][0], sml[3][c][0]));
        const float f = m[rt] == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m[rt] - mm);
        float* dst = so + (wave * 16 + i) * OS;
#pragma unroll
        for (int cc = 0; cc < G::NCH; ++cc)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e4 = 0; e4 < G::CH; e4 += 4) {
              const int tt = cc * G::CH + e4;
              *reinterpret_cast<float4*>(dst + cc * 16 * G::CH + G::CH * (4 * g + r) + e4) =
                  make_float4(o[rt][tt][r] * f, o[rt][tt + 1][r] * f, o[rt][tt + 2][r] * f, o[rt][tt + 3][r] * f);
            }
        __syncthreads();
        for (int idx = tid; idx < 16 * (D / 4); idx += 256) {
          const int row = idx / (D / 4), c4 = idx % (D / 4), r = (rb * RT + rt) * 16 + row;
          if (r >= rows) continue;
          float M = NEG_INF, L = 0.f;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 4; ++w) M = fmaxf(M, sml[w][rt * 16 + row][0]);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float mw = sml[w][rt * 16 + row][0];
            L += sml[w][rt * 16 + row][1] * (mw == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(mw - M));
            const float4 v = *reinterpret_cast<const float4*>(so + (w * 16 + row) * OS + 4 * c4);
            a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
          }
          if (whole) {
            put_row<D>(p, sq.q0, h, r, c4, a, M, L, vs);
          } else {
            const long at = (long)slot * (RT * 16) + rt * 16 + row;
            *reinterpret_cast<float4*>(p.part_o + at * D + 4 * c4) = a;
            if (c4 == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(M, L);
          }
        }
        __syncthreads();
      }
    }
    if (!whole && t0 == 0 && tid == 0) {
      const int last = (cur + sq.steps - 1) / per;  // workgroup that holds the unit's last step
      *reinterpret_cast<int4*>(p.desc + 4 * wg) = make_int4(last - wg + 1, b, h, rb);
    }
    cur += t1 - t0;
  }
}

// Joins the pieces of a unit cut between workgroups: grid (workgroups, row groups of 4), a
// wave a row, lanes over the values and, where they are fewer than 64 x 4, over the pieces.
template <int D>
__global__ __launch_bounds__(256) void k_tree_combine(TreeAttnParams p, int block_rows) {
  const int wg = blockIdx.x;
  const int4 ds = *reinterpret_cast<const int4*>(p.desc + 4 * wg);
  if (ds.x == 0) return;
  constexpr int CL = D / 4, PG = 64 / CL;  // lanes over a row's values, groups of lanes over the pieces
  const int lane = threadIdx.x & 63, row = blockIdx.y * 4 + (threadIdx.x >> 6);
  const int q0 = p.q_indptr[ds.y], rows = (p.q_indptr[ds.y + 1] - q0) * p.group;
  const int r = ds.w * block_rows + row;
  if (row >= block_rows || r >= rows) return;
  auto slot = [&](int k) { return (long)(k == 0 ? 2 * wg + 1 : 2 * (wg + k)) * block_rows + row; };
  float M = NEG_INF;
  for (int k = lane; k < ds.x; k += 64) M = fmaxf(M, p.part_ml[2 * slot(k)]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) M = fmaxf(M, __shfl_xor(M, d));
  const int c4 = lane % CL, pg = lane / CL;
  float L = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = pg; k < ds.x; k += PG) {
    const long at = slot(k);
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * c4);
    const float f = ml.x == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(ml.x - M);
    L += ml.y * f;
    a.x += v.x * f; a.y += v.y * f; a.z += v.z * f; a.w += v.w * f;
  }
#pragma unroll
  for (int d = CL; d < 64; d <<= 1) {
    L += __shfl_xor(L, d);
    a.x += __shfl_xor(a.x, d); a.y += __shfl_xor(a.y, d); a.z += __shfl_xor(a.z, d); a.w += __shfl_xor(a.w, d);
  }
  if (pg) return;
  const float vs = p.v_scale ? p.v_scale[ds.z] : 1.f;
  put_row<D>(p, q0, ds.z, r, c4, a, M, L, vs);
}

// Bit i of row t: drafted token i is t or one of its ancestors.  One thread a token; a parent
// comes before its child, so the walk ends.
__global__ __launch_bounds__(256) void k_tree_mask(const int* parents, const int* q_indptr, int B, int T, int max_q,
                                                   int words, uint64_t* mask, int* status) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= T) return;
  int lo = 0, hi = B;  // last sequence with q_indptr[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q_indptr[mid] <= t) lo = mid; else hi = mid;
  }
  const int q0 = q_indptr[lo];
  for (int w = 0; w < words; ++w) mask[(long)t * words + w] = 0;
  int j = t - q0;
  if (q0 < 0 || j < 0 || j >= max_q) {
    if (status) or_agent(status, ST_LENGTH);
    return;
  }
  for (;;) {
    mask[(long)t * words + (j >> 6)] |= 1ull << (j & 63);
    const int up = parents[q0 + j];
    if (up < 0) break;
    if (up >= j) {
      if (status) or_agent(status, ST_PARENT);
      break;
    }
    j = up;
  }
}

template <int D, int RT, bool FP8>
void launch_one(const TreeAttnParams& p, hipStream_t s) {
  constexpr int OCC = RT == 1 && D <= 128 ? 2 : 1;
  hipLaunchKernelGGL((k_tree_attention<D, RT, FP8, OCC>), dim3(p.n_wg), dim3(256), (p.B + 1) * sizeof(int), s, p);
}

template <int D>
hipError_t launch_d(const TreeAttnParams& p, const TreeAttnPlan& pl, bool fp8, hipStream_t s) {
  switch (pl.row_tiles) {
    case 1: fp8 ? launch_one<D, 1, true>(p, s) : launch_one<D, 1, false>(p, s); break;
    default:
      if constexpr (D <= 128) fp8 ? launch_one<D, 2, true>(p, s) : launch_one<D, 2, false>(p, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int rows = min(pl.row_tiles * 16, p.max_q * p.group);
  hipLaunchKernelGGL(k_tree_combine<D>, dim3(p.n_wg, (rows + 3) / 4), dim3(256), 0, s, p, pl.row_tiles * 16);
  return hipGetLastError();
}

}  // namespace

TreeAttnPlan tree_attn_plan(int D, int rows) {
  TreeAttnPlan pl;
  pl.row_tiles = rows <= 16 || D > 128 ? 1 : 2;
  pl.n_wg = pl.row_tiles == 1 && D <= 128 ? 512 : 256;
  const size_t slots = 2 * (size_t)pl.n_wg, r = (size_t)pl.row_tiles * 16;
  pl.desc_bytes = (size_t)pl.n_wg * 16;
  pl.ml_bytes = slots * r * 8;
  pl.o_bytes = slots * r * D * 4;
  return pl;
}

hipError_t launch_tree_attention(const TreeAttnParams& p, const TreeAttnPlan& pl, int D, bool fp8, hipStream_t s) {
  switch (D) {
    case 64: return launch_d<64>(p, pl, fp8, s);
    case 128: return launch_d<128>(p, pl, fp8, s);
    default: return launch_d<256>(p, pl, fp8, s);
  }
}

hipError_t launch_tree_mask(const int* parents, const int* q_indptr, int B, int T, int max_q, int words, uint64_t* mask,
                            int* status, hipStream_t s) {
  hipLaunchKernelGGL(k_tree_mask, dim3((T + 255) / 256), dim3(256), 0, s, parents, q_indptr, B, T, max_q, words, mask, status);
  return hipGetLastError();
}

}  // namespace lora
