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
// Split: the keys of all (sequence, kv head, row block) units form one line of steps; a
// workgroup's stretch of it is found, whatever the sequences' lengths, from a prefix sum over
// the sequences that every workgroup computes itself (find_stretch), so the host needs no
// lengths.  A unit cut between workgroups leaves its pieces (m, l, unnormalised O in
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

__device__ __forceinline__ uint4 signed_q(const uint4& v, uint32_t flip) {
  return make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
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
// drafted token j of n sees.  Its mask row: of one word, from LDS (`own`, the sequence's rows;
// a load from memory would wait for every key and value in flight, which return in order), of
// more from memory; without a mask, the causal rule.
__device__ __forceinline__ uint32_t visible8(const TreeAttnParams& p, const uint64_t* own, int q0, int j, int d0, int n) {
  if (d0 <= -8) return 0xffu;
  if (d0 >= n) return 0u;
  uint32_t bits;
  if (!p.mask) {
    const int c = j - d0 + 1;
    bits = c >= 8 ? 0xffu : c <= 0 ? 0u : (1u << c) - 1u;
  } else {
    const int first = max(d0, 0), w = first >> 6, o = first & 63;
    uint64_t v;
    if (p.words == 1) {
      v = own[j] >> o;
    } else {
      const uint64_t* row = p.mask + (long)(q0 + j) * p.words;
      v = row[w] >> o;
      if (o > 56 && w + 1 < p.words) v |= row[w + 1] << (64 - o);
    }
    bits = (uint32_t)v;
    if (d0 < 0) bits = (bits << -d0) | ((1u << -d0) - 1u);
  }
  const int keep = n - d0;
  if (keep < 8) bits &= (1u << keep) - 1u;
  return bits & 0xffu;
}

// What a step of a unit counts on the line.  Where waves share the keys (SHARED, 128 rows a block)
// a step of 64 rows or fewer takes them less time: 2.1 to 2.6 us against 3.5 (16 sequences with trees
// of up to 64 tokens over up to 2,048 keys, 8-bit cache: 42.5 us with all steps alike, 36.5 so).  How much
// less depends on the cache and the heads; one weight for all is a compromise.  16 other sequences with
// trees, calls in us, all alike and so: trees of up to 64, 8-bit cache, heads of 64 37.1 and 35.7, of
// 128 56.4 and 58.1, of 256 97.2 and 94.4, 16-bit 41.7 and 43.3, 49.6 and 53.3, 95.5 and 100.6; trees of 16,
// 16-bit, 21.8 and 21.7, 29.2 and 29.8, 61.4 and 55.8, 8-bit within 0.3.
constexpr int FULL = 3, HALF_FULL = 2;
template <bool SHARED>
__device__ __forceinline__ int step_weight(int rows) { return !SHARED ? 1 : rows > 64 ? FULL : HALF_FULL; }

// One sequence: its queries and keys, its steps, row blocks (the last one's steps count `last`),
// and what the steps of one kv head's units count together.
struct Seq { int q0, n, kv, steps, blocks, last, head, bad; };  // bad: EMPTY, LEFT_OUT
enum { EMPTY = 1, LEFT_OUT = 2 };
// Steps of row block rb of 128 rows, and of the blocks before it.  In order, `group` blocks hold 128
// tokens, so that every `group` blocks a block's last token sees a step more.
__device__ __forceinline__ bool in_order(const TreeAttnParams& p, const Seq& s) { return p.counted && s.kv >= s.n; }
__device__ __forceinline__ int first_steps(const Seq& s) { return (s.kv - s.n + ATTN_KEYS - 1) / ATTN_KEYS + 1; }
__device__ __forceinline__ int steps_of(const TreeAttnParams& p, const Seq& s, int rb) {
  return in_order(p, s) ? min(s.steps, first_steps(s) + rb / p.group) : s.steps;
}
__device__ __forceinline__ int steps_before(const TreeAttnParams& p, const Seq& s, int rb) {
  if (!in_order(p, s)) return rb * s.steps;
  const int first = first_steps(s), m = rb / p.group;
  return p.group * (m * first + m * (m - 1) / 2) + (rb - m * p.group) * min(s.steps, first + m);
}
// The row block that step x of a kv head's blocks is in.
__device__ __forceinline__ int block_at(const TreeAttnParams& p, const Seq& s, int x) {
  if (!in_order(p, s)) return x / s.steps;
  int m = 0;
  while ((m + 1) * p.group < s.blocks && steps_before(p, s, (m + 1) * p.group) <= x) ++m;
  return m * p.group + (x - steps_before(p, s, m * p.group)) / steps_of(p, s, m * p.group);
}

// Whether a sequence's rows [q0, q1) lie in the call's and are not more than it allows for.
__device__ __forceinline__ bool tokens_fit(int q0, int q1, int T, int max_q) {
  return q0 >= 0 && q1 >= q0 && q1 <= T && q1 - q0 <= max_q;
}

template <bool SHARED>
__device__ __forceinline__ Seq make_seq(const TreeAttnParams& p, int q0, int q1, int kv, int block_rows) {
  Seq s;
  s.q0 = q0;
  s.kv = kv;
  s.bad = 0;
  s.n = q1 - q0;
  if (!tokens_fit(q0, q1, p.T, p.max_q)) { s.n = 0; s.bad = LEFT_OUT; }
  if (kv < s.n || (long)kv > ((long)p.max_pages << p.page_log2)) { s.kv = 0; s.bad |= EMPTY; }
  s.steps = max(1, (s.kv + ATTN_KEYS - 1) / ATTN_KEYS);
  s.blocks = (s.n * p.group + block_rows - 1) / block_rows;
  s.last = step_weight<SHARED>(s.n * p.group - (s.blocks - 1) * block_rows);
  const int full = s.blocks - 1;
  if (s.blocks == 0) s.head = 0;
  else if (SHARED) s.head = FULL * steps_before(p, s, full) + s.last * steps_of(p, s, full);
  else s.head = s.steps * s.blocks;
  return s;
}

// A workgroup's stretch [cur, end) of the line of all units' steps, `per` of it a workgroup, and
// the sequence it begins in, from a prefix sum over the sequences' work that leaves cum[b], what
// lies before sequence b, in LDS.  (Cutting every unit evenly instead, so that nobody begins a
// second one, took a search that cost what it saved.)  `loose`: rows that no sequence has (LOOSE),
// some of them perhaps between sequences (LEFT_OUT), or all (NO_ROWS).
struct Stretch { int cur, end, per, b, loose; Seq first; };
enum { LOOSE = 1, NO_ROWS = 4 };
template <int THREADS, bool SHARED>
__device__ __forceinline__ Stretch find_stretch(const TreeAttnParams& p, int wg, int block_rows, int* cum, int2* wave_sum,
                                                Stretch* found) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, each = (p.B + THREADS - 1) / THREADS;
  uint32_t mine = 0;  // the line's length has 31 bits, unless offsets give rows to several sequences
  int loose = 0;
  Seq s{};
  for (int i = 0; i < each; ++i) {
    const int b = tid * each + i;
    if (b < p.B) {
      const int q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1];
      s = make_seq<SHARED>(p, q0, q1, p.kv_len[b], block_rows);
      const bool ends = (b == 0 && q0 != 0) || (b == p.B - 1 && q1 != p.T);
      if ((s.bad || ends) && blockIdx.x == 0 && p.status) or_agent(p.status, ST_LENGTH);
      loose |= (s.bad & LEFT_OUT) | (ends ? LOOSE : 0);
      mine += (uint32_t)(p.n_kv * s.head);
      cum[b + 1] = (int)mine;
    }
  }
  loose = (__any(loose & LOOSE) ? LOOSE : 0) | (__any(loose & LEFT_OUT) ? LEFT_OUT : 0);
  uint32_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t u = __shfl_up(incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 63) wave_sum[wave] = make_int2((int)incl, loose);
  if (tid == 0) {
    cum[0] = 0;
    found->cur = found->end = 0;  // for a workgroup past the end
  }
  __syncthreads();
  uint32_t ahead = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    const int2 u = wave_sum[w];
    ahead += w < wave ? (uint32_t)u.x : 0u;
    all += (uint32_t)u.x;
    loose |= u.y;
  }
  if (loose & LEFT_OUT) {
    // Descending offsets can give rows to several sequences, and the line more steps than the host
    // has allowed for T rows: with more rows than T in all, every sequence is left out.
    int rows = 0;
    for (int i = 0; i < each; ++i) {
      const int b = tid * each + i;
      if (b >= p.B) continue;
      const int q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1];
      rows += tokens_fit(q0, q1, p.T, p.max_q) ? q1 - q0 : 0;  // 4,096 times 65,536 at most
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) rows += __shfl_xor(rows, d);
    __syncthreads();  // the sums are read
    if (lane == 0) wave_sum[wave].x = rows;
    __syncthreads();
    rows = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) rows += wave_sum[w].x;
    if (rows > p.T) return Stretch{0, 0, 1, 0, LEFT_OUT | NO_ROWS, Seq{}};
  }
  int before = (int)ahead;
  const int total = (int)all;
  // a step at least: a shorter stretch inside a unit may hold the beginning of none
  const int per = max((total + p.n_wg - 1) / p.n_wg, step_weight<SHARED>(min(p.max_q * p.group, block_rows)));
  const int cur = min(total, wg * per), end = min(total, cur + per);
  int from = before;
  for (int i = 0; i < each; ++i) {
    const int b = tid * each + i;
    if (b < p.B) {
      const int next = before + cum[b + 1];
      if (from <= cur && cur < next) {
        if (each > 1) s = make_seq<SHARED>(p, p.q_indptr[b], p.q_indptr[b + 1], p.kv_len[b], block_rows);
        *found = Stretch{cur, end, per, b, 0, s};
      }
      cum[b + 1] = next;
      from = next;
    }
  }
  __syncthreads();
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  return Stretch{uniform(found->cur), uniform(found->end), uniform(found->per), uniform(found->b), uniform(loose),
                 Seq{uniform(found->first.q0), uniform(found->first.n), uniform(found->first.kv), uniform(found->first.steps),
                     uniform(found->first.blocks), uniform(found->first.last), uniform(found->first.head), 0}};
}

// Rows that no sequence has: out 0, lse -inf.  Each workgroup takes its share of all rows.  Unless a
// sequence was left out they lie before the first one's and behind the last one's.
template <int D, int THREADS>
__device__ __forceinline__ void clear_loose(const TreeAttnParams& p, int wg, int loose) {
  const int lo = p.q_indptr[0], hi = p.q_indptr[p.B];
  for (int t = wg; t < p.T; t += p.n_wg) {
    bool none = t < lo || t >= hi || (loose & NO_ROWS);
    if ((loose & LEFT_OUT) && !(loose & NO_ROWS)) {
      int taken = 0;
      for (int b = threadIdx.x; b < p.B; b += THREADS) {
        const int q0 = p.q_indptr[b], q1 = p.q_indptr[b + 1];
        taken |= tokens_fit(q0, q1, p.T, p.max_q) && q0 <= t && t < q1;
      }
      none = !__syncthreads_or(taken);
    }
    if (!none) continue;
    uint4* row = reinterpret_cast<uint4*>(p.out + (long)t * p.n_q * D);
    for (int c = threadIdx.x; c < p.n_q * (D / 8); c += THREADS) row[c] = zero4();
    if (p.lse)
      for (int h = threadIdx.x; h < p.n_q; h += THREADS) p.lse[(long)t * p.n_q + h] = NEG_INF;
  }
}

// Waits until products that may still be writing these accumulators have written them.  The compiler
// keeps that distance for instructions that it knows, not for ones in assembly: 24 wait states are
// more than any product here takes.  Tied to the accumulators, so that their products come before.
template <int NT>
__device__ __forceinline__ void settle(v4f (&o)[NT]) {
  if constexpr (NT == 4) {
    asm volatile("s_nop 15\n\ts_nop 7" : "+v"(o[0]), "+v"(o[1]), "+v"(o[2]), "+v"(o[3]));
  } else {
    static_assert(NT % 8 == 0, "tiles by the eight");
#pragma unroll
    for (int t = 0; t < NT; t += 8)
      asm volatile("s_nop 15\n\ts_nop 7"
                   : "+v"(o[t]), "+v"(o[t + 1]), "+v"(o[t + 2]), "+v"(o[t + 3]), "+v"(o[t + 4]), "+v"(o[t + 5]), "+v"(o[t + 6]), "+v"(o[t + 7]));
  }
}

// The scores of 32 keys of COUNT row tiles (S^T: lane (g, i) has keys 8 g .. 8 g + 7 of row i)
// into the running softmax; pb: the probabilities as the MFMA operand of O^T = V^T P^T.
// m, l, o: the first of the tiles'.
template <int NT, int COUNT, bool SPECIAL>
__device__ __forceinline__ void softmax_step(const v4f (&s)[COUNT][2], float sc, const uint32_t (&vis)[COUNT], float* m, float* l,
                                             v4f (*o)[NT], uint4 (&pb)[COUNT]) {
  float x[COUNT][8], mx[COUNT];  // products of keys 8 g + e; sc >= 0 takes them to log2 units
  bool over = false;
#pragma unroll
  for (int c = 0; c < COUNT; ++c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[c][e] = SPECIAL && !((vis[c] >> e) & 1u) ? NEG_INF : s[c][e >> 2][e & 3];
    mx[c] = fmaxf(fmaxf(fmaxf(x[c][0], x[c][1]), x[c][2]), fmaxf(fmaxf(x[c][3], x[c][4]), fmaxf(fmaxf(x[c][5], x[c][6]), x[c][7]))) * sc;
    over |= mx[c] > m[c] + SLACK;
  }
  if (__any(over)) {
#pragma unroll
    for (int c = 0; c < COUNT; ++c) {
      mx[c] = fmaxf(mx[c], __shfl_xor(mx[c], 16));
      mx[c] = fmaxf(mx[c], __shfl_xor(mx[c], 32));
      // each row by its own scores alone: what a row gets does not depend on its neighbours
      const bool up = mx[c] > m[c] + SLACK;
      const float f = up ? __builtin_amdgcn_exp2f(m[c] - mx[c]) : 1.f;
      m[c] = up ? mx[c] : m[c];
      l[c] *= f;
      // in place, by hand: the compiler multiplies into other registers, and then has the way
      // around this branch, every step's, copy all of o (32 sequences of 2,048 keys, 256 rows, 8-bit
      // cache: 139 us against 130)
      settle<NT>(o[c]);
#pragma unroll
      for (int tt = 0; tt < NT; ++tt)
#pragma unroll
        for (int r = 0; r < 4; ++r) asm("v_mul_f32 %0, %1, %0" : "+v"(o[c][tt][r]) : "v"(f));
    }
  }
#pragma unroll
  for (int c = 0; c < COUNT; ++c) {
    const float ref = m[c] == NEG_INF ? 0.f : m[c];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[c][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[c][e], sc, -ref));
      if (SPECIAL && !((vis[c] >> e) & 1u)) x[c][e] = 0.f;  // with a scale of 0, -inf * 0 is no zero
    }
    l[c] += ((x[c][0] + x[c][1]) + (x[c][2] + x[c][3])) + ((x[c][4] + x[c][5]) + (x[c][6] + x[c][7]));
    // P enters the MFMA in bf16 (relative error 2^-8 an element at most, as the output's own
    // rounding); its sum l is taken before the rounding, in 32 bits
    pb[c] = make_uint4(bf16x2_rne(x[c][0], x[c][1]), bf16x2_rne(x[c][2], x[c][3]), bf16x2_rne(x[c][4], x[c][5]), bf16x2_rne(x[c][6], x[c][7]));
  }
}

// 8 keys x 2 values in VE-word rows -> the MFMA operand of one value: word w of the rows, its
// low or high half by `odd`.
template <int VE>
__device__ __forceinline__ uint4 transposed(const uint32_t (&vb)[8][VE], int w, int odd) {
  const uint32_t sel = odd ? 0x07060302u : 0x05040100u;
  return make_uint4(__builtin_amdgcn_perm(vb[1][w], vb[0][w], sel), __builtin_amdgcn_perm(vb[3][w], vb[2][w], sel),
                    __builtin_amdgcn_perm(vb[5][w], vb[4][w], sel), __builtin_amdgcn_perm(vb[7][w], vb[6][w], sel));
}

// A lane's V words of one key, widened to bf16.
template <typename G, bool FP8>
__device__ __forceinline__ void widen_v(const uint32_t* in, uint32_t* out) {
  if constexpr (FP8) {
#pragma unroll
    for (int w = 0; w < G::NCH * G::VW; ++w) {
      const uint2 u = fp8x4_to_bf16(in[w]);
      out[2 * w] = u.x;
      out[2 * w + 1] = u.y;
    }
  } else {
#pragma unroll
    for (int w = 0; w < G::NCH * G::VW; ++w) out[w] = in[w];
  }
}

// K operand of MFMA step st from a lane's loads of 16 keys.
template <bool FP8>
__device__ __forceinline__ uint4 k_operand(const uint4* kr, int st) {
  if constexpr (FP8) {
    const uint4 w = kr[st >> 1];
    const uint2 lo = fp8x4_to_bf16((st & 1) ? w.z : w.x), hi = fp8x4_to_bf16((st & 1) ? w.w : w.y);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else {
    return kr[st];
  }
}

// V rows (as loaded) of a group of 32 keys made safe for a product that multiplies unseen keys by zero:
// rows of keys past the end, and of pages that do not exist, hold anything and are zeroed; a
// drafted key that only some rows see must not reach the others through 0 * NaN, so rows with
// values that are not finite are zeroed too, and returned (bit e: key 8 g + e of this lane's
// group g) to be added apart, to the rows that see them (add_odd_keys).
template <bool FP8, int W>
__device__ __forceinline__ uint32_t clean_v(uint32_t (&row)[8][W], int g, bool gone, int d0, int n) {
  // a value that is not finite has all its exponent bits (e4m3: all but the sign), to which
  // adding one carries into the sign's place
  constexpr uint32_t BITS = FP8 ? 0x7f7f7f7fu : 0x7f807f80u, ONE = FP8 ? 0x01010101u : 0x00800080u, CARRY = FP8 ? 0x80808080u : 0x80008000u;
  uint32_t odd = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool none = gone || d0 + e >= n;
    uint32_t carry = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      row[e][w] = none ? 0u : row[e][w];
      carry |= (row[e][w] & BITS) + ONE;
    }
    const uint64_t any = __ballot((carry & CARRY) != 0);
    if ((any >> (16 * g)) & 0xffffu) {
      odd |= 1u << e;
#pragma unroll
      for (int w = 0; w < W; ++w) row[e][w] = 0u;
    }
  }
  return odd;
}

// The keys that clean_v took out (bit 8 g + e of `odd`), one at a time: each as the operand
// whose only key it is, its product added to the rows that see it.  In part `part` of PARTS of
// the tiles of O^T, where the rows were cleaned in parts.
template <int D, bool FP8, int PARTS = 1>
__device__ __forceinline__ void add_odd_keys(uint32_t odd, const char* v0, const char* v1, const uint4& pb, uint32_t vis,
                                             v4f (&o)[D / 16], int part = 0) {
  using G = Geo<D, FP8>;
  constexpr int VE = G::NCH * G::CH / 2;
  const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  for (int kk = 0; kk < 32; ++kk) {
    if (!((odd >> kk) & 1u)) continue;
    const int gk = kk >> 3, e = kk & 7;
    const char* row = (gk < 2 ? v0 : v1) + (kk & 15) * G::ROWB + i * G::VB;
    uint32_t raw[G::NCH * G::VW], v[VE];
#pragma unroll
    for (int c = 0; c < G::NCH; ++c) ldg_words<G::VB>(row + c * 16 * G::VB, &raw[c * G::VW]);
    widen_v<G, FP8>(raw, v);
    const bool sees = (__shfl((int)vis, 16 * gk + i) >> e) & 1;
#pragma unroll
    for (int tt = 0; tt < D / 16; ++tt) {
      if (PARTS > 1 && tt / (D / 16 / PARTS) != part) continue;
      const uint32_t half = (v[tt >> 1] >> (16 * (tt & 1))) & 0xffffu;
      const uint32_t val = g == gk ? half << (16 * (e & 1)) : 0u;
      const uint4 a = make_uint4((e >> 1) == 0 ? val : 0u, (e >> 1) == 1 ? val : 0u, (e >> 1) == 2 ? val : 0u, (e >> 1) == 3 ? val : 0u);
      const v4f add = mfma_bf16_16x16x32(a, pb, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int r = 0; r < 4; ++r) o[tt][r] += sees ? add[r] : 0.f;
      __builtin_amdgcn_sched_barrier(0);  // one tile at a time: this path is rare, its registers are not
    }
  }
}

// What the join needs of a unit that workgroup wg began and others ended: its pieces, first
// query row, rows, kv head and row block.
__device__ __forceinline__ void put_desc(const TreeAttnParams& p, int wg, int pieces, const Seq& sq, int h, int rb) {
  int4* d = reinterpret_cast<int4*>(p.desc + ATTN_DESC * wg);
  d[0] = make_int4(pieces, sq.q0, sq.n * p.group, h);
  d[1] = make_int4(rb, 0, 0, 0);
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

// Write the finished rows of a tile in the lanes' layout: lane (g, i) has row r at places
// 16 CH c + CH (4 g + x) + e of tile c CH + e, element x.
template <int D, int CH>
__device__ __forceinline__ void put_tile(const TreeAttnParams& p, int q0, int rows, int h, int r, int g, const v4f (&o)[D / 16],
                                         float M, float L, float vs) {
  if (r >= rows) return;
  const float inv = L == 0.f ? 0.f : vs / L;
  const int j = r / p.group;
  const long at = (long)(q0 + j) * p.n_q + h * p.group + (r - j * p.group);
#pragma unroll
  for (int c = 0; c < D / (16 * CH); ++c)
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int e = 0; e < CH; e += 4) {
        const int t = c * CH + e;
        *reinterpret_cast<uint2*>(p.out + at * D + 16 * CH * c + CH * (4 * g + x) + e) =
            make_uint2(bf16x2_rne(o[t][x] * inv, o[t + 1][x] * inv), bf16x2_rne(o[t + 2][x] * inv, o[t + 3][x] * inv));
      }
  if (g == 0 && p.lse) p.lse[at] = L == 0.f ? NEG_INF : (M + __builtin_amdgcn_logf(L)) * 0.69314718055994531f;
}

// Few rows: four waves split a step's 128 keys.  Bound by HBM: 64 sequences of up to 8,192 keys in
// 16 bits, 4 rows a kv head (922 MB), 166 us, 5.5 TB/s; one of 131,072 in 8 bits 51 us, 5.3 TB/s.
// Short work is bound by latencies: of the 16.6 us for 16 sequences of 1,024 keys (67 MB) the first
// 4 pass before keys are on their way (the launch, the prefix sum, the page table, the queries).
template <int D, int RT, bool FP8, int OCC>
__global__ __launch_bounds__(256, OCC) void k_tree_attention(TreeAttnParams p) {
  using G = Geo<D, FP8>;
  constexpr int NT = D / 16;       // 16-row tiles of O^T
  constexpr int OS = D + 4;        // row stride of the joining buffer (floats)
  __shared__ __attribute__((aligned(16))) float so[4 * 16 * OS];
  __shared__ float sml[4][RT * 16][2];
  __shared__ int2 wave_sum[4];
  __shared__ Stretch found;
  __shared__ uint64_t smask[64];  // the sequence's masks, where they are of one word
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

  const Stretch mine = find_stretch<256, false>(p, wg, RT * 16, cum, wave_sum, &found);
  if (tid == 0) p.desc[ATTN_DESC * wg] = 0;
  if (mine.loose) clear_loose<D, 256>(p, wg, mine.loose);
  int cur = mine.cur, b = mine.b;
  Seq sq = mine.first;
  const int end = mine.end;

  const int page = 1 << p.page_log2;
  const int koff = (8 * ((i >> 2) & 1) + (i & 3)) * G::ROWB + 16 * g;
  const int voff = 8 * (g & 1) * G::ROWB + i * G::VB;

  while (cur < end) {
    while (__builtin_amdgcn_readfirstlane(cum[b + 1]) <= cur) ++b;  // skips sequences without queries
    if (b != mine.b) sq = make_seq<false>(p, ld_table(p.q_indptr + b), ld_table(p.q_indptr + b + 1), ld_table(p.kv_len + b), RT * 16);
    const int local = cur - __builtin_amdgcn_readfirstlane(cum[b]);
    const int unit = local / sq.steps, t0 = local - unit * sq.steps;
    const int t1 = min(sq.steps, t0 + end - cur);
    const int h = unit / sq.blocks, rb = unit - h * sq.blocks;
    const int rows = sq.n * p.group, prefix = sq.kv - sq.n, kv = sq.kv;
    const int* table = p.page_table + (long)b * p.max_pages;

    // scores in log2 units; a negative scale is taken as the queries' sign
    const float scale = FP8 ? p.scale_log2 * p.k_scale[h] : p.scale_log2, sc = fabsf(scale);
    const uint32_t flip = scale < 0.f ? 0x80008000u : 0u;
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
        for (int s = wave; s < G::KS; s += 4) sq_ops[s][lane] = r < rows ? signed_q(ldg16(src + q_place<FP8>(s, g)), flip) : zero4();
      } else {
#pragma unroll
        for (int s = 0; s < G::KS; ++s) q[rt][s] = r < rows ? signed_q(ldg16(src + q_place<FP8>(s, g)), flip) : zero4();
      }
    }
    const bool masks = p.mask && p.words == 1;
    if (masks && tid < sq.n) smask[tid] = p.mask[sq.q0 + tid];  // words 1: n <= 64
    if (Q_LDS || masks) __syncthreads();

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
          const uint4 a = k_operand<FP8>(kr[kt], st);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) s[rt][kt] = mfma_bf16_16x16x32(a, Q_LDS ? qs : q[rt][Q_LDS ? 0 : st], s[rt][kt]);
        }
      }
      if (!SPECIAL && more) load_k(nb0, nb1);

      const int d0 = key0 + 8 * g - prefix;  // draft place of this lane's 8 keys
      const bool gone = g < 2 ? bad0 : bad1;
      uint4 pb[RT];
      uint32_t vis[RT] = {};
      if constexpr (SPECIAL) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) vis[rt] = gone ? 0u : visible8(p, smask, sq.q0, jrow[rt], d0, sq.n);
      }
      softmax_step<NT, RT, SPECIAL>(s, sc, vis, m, l, o, pb);

      // V: 8 keys x CH values a lane, widened to bf16
      uint32_t odd = 0;
      if constexpr (SPECIAL) {
        const uint32_t mine = clean_v<FP8>(vr, g, gone, d0, sq.n);
#pragma unroll
        for (int gk = 0; gk < 4; ++gk) odd |= (uint32_t)__builtin_amdgcn_readlane((int)mine, 16 * gk) << (8 * gk);
      }
      uint32_t vb[8][VE];
#pragma unroll
      for (int e = 0; e < 8; ++e) widen_v<G, FP8>(vr[e], vb[e]);
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) {
        const uint4 a = transposed<VE>(vb, tt >> 1, tt & 1);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) o[rt][tt] = mfma_bf16_16x16x32(a, pb[rt], o[rt][tt]);
      }
      if constexpr (SPECIAL) {
        const char* vc = reinterpret_cast<const char*>(p.v_cache);
        if (odd)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) add_odd_keys<D, FP8>(odd, vc + b0, vc + b1, pb[rt], vis[rt], o[rt]);
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
      put_desc(p, wg, (cur + sq.steps - 1) / mine.per - wg + 1, sq, h, rb);
    }
    cur += t1 - t0;
  }
}

// Joins the pieces of a unit cut between workgroups: grid (workgroups, row groups).  The lanes
// of a wave go over a row's values and, where those are fewer than 64 x 4, over the pieces; the
// four waves take a row each, or with WIDE a row's pieces in turn.  A chain of latencies, a launch's
// among them: 4.0 us for 4 pieces a unit, 5.9 for the 64 pieces of one long sequence.  (Joining in
// the workgroup that finishes a unit last needs its pieces written through to memory, and counters:
// slower on every case that was measured.)
template <int D, bool WIDE>
__global__ __launch_bounds__(256) void k_tree_combine(TreeAttnParams p, int block_rows) {
  const int wg = blockIdx.x;
  const int4 ds = *reinterpret_cast<const int4*>(p.desc + ATTN_DESC * wg);
  const int rb = p.desc[ATTN_DESC * wg + 4];
  if (ds.x == 0) return;
  constexpr int CL = D / 4;                        // lanes over a row's values
  constexpr int PW = 64 / CL, PG = PW * (WIDE ? 4 : 1);  // groups of lanes over the pieces: a wave's, all
  __shared__ float4 so[WIDE ? 4 : 1][CL];
  __shared__ float2 sml[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = WIDE ? blockIdx.y : blockIdx.y * 4 + wave;
  const int r = rb * block_rows + row;
  if (row >= block_rows || r >= ds.z) return;  // WIDE: the whole workgroup
  auto slot = [&](int k) { return (long)(k == 0 ? 2 * wg + 1 : 2 * (wg + k)) * block_rows + row; };
  const int c4 = lane % CL, pg = lane / CL + (WIDE ? PW * wave : 0);
  float M = NEG_INF, L = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  // eight pieces a round with a running maximum: all of a round's loads are in flight together
  for (int k0 = pg; k0 < ds.x; k0 += 8 * PG) {
    float2 ml[8];
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const long at = slot(min(k0 + k * PG, ds.x - 1));  // the last piece again, with no weight
      ml[k] = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
      v[k] = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * c4);
    }
    float mn = M;
#pragma unroll
    for (int k = 0; k < 8; ++k) mn = fmaxf(mn, ml[k].x);
    const float back = M == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(M - mn);
    L *= back; a.x *= back; a.y *= back; a.z *= back; a.w *= back;
    M = mn;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // selected, not branched around: a branch would pull the loads apart, one wait each
      const bool real = k0 + k * PG < ds.x;
      const float f = ml[k].x == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(ml[k].x - M);
      L += real ? ml[k].y * f : 0.f;
      a.x += real ? v[k].x * f : 0.f; a.y += real ? v[k].y * f : 0.f; a.z += real ? v[k].z * f : 0.f; a.w += real ? v[k].w * f : 0.f;
    }
  }
  {  // the groups of lanes hold other pieces of the same row
    float mn = M;
#pragma unroll
    for (int d = CL; d < 64; d <<= 1) mn = fmaxf(mn, __shfl_xor(mn, d));
    const float f = M == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(M - mn);
    L *= f; a.x *= f; a.y *= f; a.z *= f; a.w *= f;
    M = mn;
  }
#pragma unroll
  for (int d = CL; d < 64; d <<= 1) {
    L += __shfl_xor(L, d);
    a.x += __shfl_xor(a.x, d); a.y += __shfl_xor(a.y, d); a.z += __shfl_xor(a.z, d); a.w += __shfl_xor(a.w, d);
  }
  if constexpr (WIDE) {
    if (lane < CL) so[wave][c4] = a;
    if (lane == 0) sml[wave] = make_float2(M, L);
    __syncthreads();
    if (wave) return;
    M = fmaxf(fmaxf(sml[0].x, sml[1].x), fmaxf(sml[2].x, sml[3].x));
    L = 0.f;
    a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = sml[w].x == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(sml[w].x - M);
      const float4 v = so[w][c4];
      L += sml[w].y * f;
      a.x += v.x * f; a.y += v.y * f; a.z += v.z * f; a.w += v.w * f;
    }
  }
  if (lane >= CL) return;
  put_row<D>(p, ds.y, ds.w, r, c4, a, M, L, p.v_scale ? p.v_scale[ds.w] : 1.f);
}

// The same for many rows (trees of many tokens times a group of heads; a prompt's chunk): eight
// waves share the keys, in rounds of up to four groups of 32.  They are loaded once for up to 128
// rows, put into LDS as MFMA operands (K and the transposed V in bf16, 1 KB a wave's read, conflict
// free; an 8-bit cache is widened once, here), and each wave takes 16 rows through all of them; of
// 64 rows or fewer, two or four waves share each 16 (32 sequences of 2,048 keys, 64 rows: 61 us
// against 70).  The next round's loads are in flight, in registers, while one is computed.
// 16 sequences with trees of up to 64 tokens over up to 2,048 keys, 8-bit cache: 36 us, 257 TFLOP/s.
// Bound by the SIMDs' instructions and waits: a round of 128 keys spends 3,650 cycles in its four
// groups (a wave's group is 256 cycles of products and about 300 of softmax, two waves a SIMD; its
// operands are 1,024 cycles of LDS reads for the eight waves), 720 in putting the next round into
// LDS and 1,900 at barriers.  Two row tiles a wave, with half the LDS reads, take as long: 2 to 4 %
// less at 32 sequences of 256 rows, 2 us more wherever units are cut, for joining the waves.  Two
// sets of operands in LDS, one barrier a round: 4 % less with 8-bit caches, 10 % more with 16-bit.
// WGS: workgroups a CU. Two, where there are units enough for twice the workgroups, fill each
// other's waits (figures at tree_attn_plan).
// A piece's slot holds O in the lanes' own layout, [row tile][x = 0 .. 3][NT / 4][lane] x 4 tiles
// of O^T, so that its stores and the join's loads are whole KBs and a wave of the join, which
// takes one x, has neighbouring values of a row.
constexpr int ROW_WAVES = 8;

template <int D, bool FP8, int WGS>
__global__ __launch_bounds__(64 * ROW_WAVES, 2 * WGS) void k_tree_attention_rows(TreeAttnParams p) {
  using G = Geo<D, FP8>;
  constexpr int NT = D / 16, BLOCK = 16 * ROW_WAVES;
  // a round's groups of 32 keys, the waves that load one, and a wave's words of a key: half a
  // group's K or V (heads of 256, and of 128 with two workgroups a CU: a quarter), 8 to 32 registers
  constexpr int GR = D * WGS >= 256 ? 2 : 4, PARTS = ROW_WAVES / GR, SW = G::NCH * G::VW / (PARTS / 2);
  static_assert(2 * G::KL / (PARTS / 2) == 2 * SW, "keys and values take the same registers");
  // V in parts: by a lane's loads of a key, or within its one load
  constexpr int LOADS = PARTS == 2 ? G::NCH : 1, LOAD_BYTES = 4 * SW / LOADS;
  constexpr int PART_BYTES = G::NCH > 1 ? 16 * G::VB : LOAD_BYTES;
  constexpr int VE = G::NCH * G::CH / 2;
  // a round's operands: K [32 keys][16 keys][MFMA step][lane], V [32 keys][tile of O^T][lane]; at
  // a unit's end, accumulators to be joined
  __shared__ uint4 ops[GR * 2 * G::KS * 64 + GR * NT * 64];
  auto sk = [&](int gr, int kt, int step) -> uint4& { return ops[((gr * 2 + kt) * G::KS + step) * 64 + (threadIdx.x & 63)]; };
  auto sv = [&](int gr, int tile) -> uint4& { return ops[GR * 2 * G::KS * 64 + (gr * NT + tile) * 64 + (threadIdx.x & 63)]; };
  __shared__ uint32_t s_odd[GR][PARTS / 2], s_bad[GR];
  __shared__ float2 sml[ROW_WAVES][16];
  __shared__ int2 wave_sum[ROW_WAVES];
  __shared__ Stretch found;
  __shared__ uint64_t smask[64];  // the sequence's masks, where they are of one word
  extern __shared__ int cum[];

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave / PARTS;                      // the 32 keys of a round this wave loads,
  const bool loads_v = wave % PARTS >= PARTS / 2;    // their values or their keys,
  const int part = wave % PARTS % (PARTS / 2);       // and which of those
  const int wg = (blockIdx.x & 7) * (p.n_wg >> 3) + (blockIdx.x >> 3);

  const Stretch mine = find_stretch<64 * ROW_WAVES, true>(p, wg, BLOCK, cum, wave_sum, &found);
  if (tid == 0) p.desc[ATTN_DESC * wg] = 0;
  if (mine.loose) clear_loose<D, 64 * ROW_WAVES>(p, wg, mine.loose);
  int cur = mine.cur, b = mine.b;
  int q0 = mine.first.q0, q1 = q0 + mine.first.n, kv_len = mine.first.kv;
  const int end = mine.end;

  const int page = 1 << p.page_log2;
  // this lane's first byte of a half of 16 keys, and which half it loads
  const int off = loads_v ? 8 * (g & 1) * G::ROWB + i * G::VB + part * PART_BYTES
                          : (8 * ((i >> 2) & 1) + (i & 3) + 4 * part) * G::ROWB + 16 * g;
  const bool second = loads_v ? g >= 2 : i >= 8;

  while (cur < end) {
    while (__builtin_amdgcn_readfirstlane(cum[b + 1]) <= cur) ++b;
    if (b != mine.b) {
      q0 = ld_table(p.q_indptr + b);
      q1 = ld_table(p.q_indptr + b + 1);
      kv_len = ld_table(p.kv_len + b);
    }
    const Seq sq = make_seq<true>(p, q0, q1, kv_len, BLOCK);
    const int local = cur - __builtin_amdgcn_readfirstlane(cum[b]);
    const int h = local / sq.head, in_head = local - h * sq.head;
    const int rb = min(block_at(p, sq, in_head / FULL), sq.blocks - 1), weight = rb == sq.blocks - 1 ? sq.last : FULL;
    // the unit's steps that begin in this stretch (of one cut inside its last step, none)
    const int steps = steps_of(p, sq, rb);
    const int in_unit = in_head - FULL * steps_before(p, sq, rb), taken = min(weight * steps - in_unit, end - cur);
    auto begun = [&](int at) { return weight == FULL ? (at + FULL - 1) / FULL : (at + HALF_FULL - 1) / HALF_FULL; };
    const int t0 = begun(in_unit), t1 = min(steps, begun(in_unit + taken));
    const bool whole = t0 == 0 && t1 == steps;
    const int slot = 2 * wg + (t0 == 0 ? 1 : 0);
    if (!whole && t0 == 0 && tid == 0) put_desc(p, wg, (cur + (steps - 1) * weight) / mine.per - wg + 1, sq, h, rb);
    cur += taken;
    if (t0 == steps) continue;
    constexpr int PER_STEP = ATTN_KEYS / ATTN_GROUP;
    const int rows = sq.n * p.group, prefix = sq.kv - sq.n;
    // without a mask no row of this block sees past its last token
    const int last_row = min(rows, (rb + 1) * BLOCK) - 1;
    const int kv = p.mask ? sq.kv : min(sq.kv, prefix + last_row / p.group + 1);
    const int* table = p.page_table + (long)b * p.max_pages;
    const int g0 = t0 * PER_STEP, g1 = min(t1 * PER_STEP, (kv + ATTN_GROUP - 1) / ATTN_GROUP);  // groups of 32 keys

    // this wave's loads of a round: V [8 keys][words], or K [load] in the same words (a second
    // round in flight measured slower: 16-token trees 19.7 us against 17.1)
    struct { uint32_t w[8][SW]; int id0, id1; } ld;
    auto fetch = [&](int t) {  // a round: up to GR groups from t on (past the last: that one again)
      const int key = min(t + grp, g1 - 1) * ATTN_GROUP;
      const int last = (sq.kv - 1) >> p.page_log2;
      ld.id0 = ld_table(table + min(key >> p.page_log2, last));
      ld.id1 = ld_table(table + min((key + 16) >> p.page_log2, last));
      auto base = [&](int id, int k) {
        const int ok = (unsigned)id < (unsigned)p.n_pages ? id : 0;
        return ((((long)ok * p.n_kv + h) << p.page_log2) + (k & (page - 1))) * G::ROWB;
      };
      const long b0 = base(ld.id0, key), b1 = base(ld.id1, key + 16);
      const char* src = reinterpret_cast<const char*>(loads_v ? p.v_cache : p.k_cache) + (second ? b1 : b0) + off;
      if (loads_v) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int c = 0; c < LOADS; ++c) ldg_words<LOAD_BYTES>(src + e * G::ROWB + c * 16 * G::VB, &ld.w[e][c * LOAD_BYTES / 4]);
      } else {
#pragma unroll
        for (int n = 0; n < 2 * SW; ++n) {  // 16-byte load n: subtile n / KL of this wave's, piece n % KL
          const uint4 w = ldg16(src + (n / G::KL) * 4 * G::ROWB + 64 * (n % G::KL));
          ld.w[4 * n / SW][4 * n % SW] = w.x; ld.w[(4 * n + 1) / SW][(4 * n + 1) % SW] = w.y;
          ld.w[(4 * n + 2) / SW][(4 * n + 2) % SW] = w.z; ld.w[(4 * n + 3) / SW][(4 * n + 3) % SW] = w.w;
        }
      }
    };
    auto stage = [&](int t) {
      const int key = min(t + grp, g1 - 1) * ATTN_GROUP;
      const bool bad0 = (unsigned)ld.id0 >= (unsigned)p.n_pages, bad1 = (unsigned)ld.id1 >= (unsigned)p.n_pages;
      if (loads_v) {
        uint32_t odd = 0;
        if (key + 32 > prefix || bad0 || bad1) {
          const uint32_t mine = clean_v<FP8>(ld.w, g, g < 2 ? bad0 : bad1, key + 8 * g - prefix, sq.n);
#pragma unroll
          for (int gk = 0; gk < 4; ++gk) odd |= (uint32_t)__builtin_amdgcn_readlane((int)mine, 16 * gk) << (8 * gk);
        }
        if (lane == 0) s_odd[grp][part] = odd;
        const int tile0 = part * (NT / (PARTS / 2));
        if constexpr (FP8) {  // a word of the eight rows at a time: four tiles
#pragma unroll
          for (int w = 0; w < SW; ++w) {
            uint32_t vb[8][2];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint2 u = fp8x4_to_bf16(ld.w[e][w]);
              vb[e][0] = u.x;
              vb[e][1] = u.y;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) sv(grp, tile0 + 4 * w + x) = transposed<2>(vb, x >> 1, x & 1);
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
#pragma unroll
          for (int tt = 0; tt < 2 * SW; ++tt) sv(grp, tile0 + tt) = transposed<SW>(ld.w, tt >> 1, tt & 1);
        }
      } else {
        uint4 kr[2 * SW];
#pragma unroll
        for (int n = 0; n < 2 * SW; ++n)
          kr[n] = make_uint4(ld.w[4 * n / SW][4 * n % SW], ld.w[(4 * n + 1) / SW][(4 * n + 1) % SW],
                             ld.w[(4 * n + 2) / SW][(4 * n + 2) % SW], ld.w[(4 * n + 3) / SW][(4 * n + 3) % SW]);
#pragma unroll
        for (int n = 0; n < 2 * SW / G::KL; ++n)
#pragma unroll
          for (int s = 0; s < G::KS; ++s) sk(grp, part + n, s) = k_operand<FP8>(kr + n * G::KL, s);
        if (lane == 0 && part == 0) {
          s_bad[grp] = (bad0 ? 1u : 0u) | (bad1 ? 2u : 0u);
          if ((bad0 || bad1) && p.status) or_agent(p.status, ST_PAGE);
        }
      }
    };
    uint64_t mask_row = 0;  // words 1: n <= 64
    if (p.mask && p.words == 1 && tid < sq.n) mask_row = p.mask[sq.q0 + tid];
    if (g0 < g1) fetch(g0);

    // scores in log2 units; a negative scale is taken as the queries' sign, a scale of 0 as queries
    // of 0 (the -inf of a key that is not seen stays -inf)
    const float scale = FP8 ? p.scale_log2 * p.k_scale[h] : p.scale_log2, sc = scale == 0.f ? 1.f : fabsf(scale);
    const uint32_t flip = scale < 0.f ? 0x80008000u : 0u;
    // Eight row tiles of 16, a wave each; of four or fewer (two or fewer), two (four) waves take
    // each, with the groups of a round between them.
    const int left = rows - rb * BLOCK, split = left <= 32 && GR == 4 ? 4 : left <= 64 ? 2 : 1;
    const int tiles = ROW_WAVES / split, tile = wave % tiles, mine_of = wave / tiles;
    // queries: column i of the tile
    const int row0 = rb * BLOCK + tile * 16;
    const bool busy = row0 < rows;
    uint4 q[G::KS];
    {
      const int r = row0 + i, j = r / p.group;
      const uint16_t* src = p.q + (long)(sq.q0 + min(j, sq.n - 1)) * p.ldq + (long)(h * p.group + (r - j * p.group)) * D;
#pragma unroll
      for (int s = 0; s < G::KS; ++s) q[s] = r < rows && scale != 0.f ? signed_q(ldg16(src + q_place<FP8>(s, g)), flip) : zero4();
    }
    v4f o[1][NT];
    float m[1] = {NEG_INF}, l[1] = {0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t) o[0][t] = v4f{0.f, 0.f, 0.f, 0.f};

    // 32 keys; `special` where they reach the drafted ones, the end or a page that does not exist
    auto group = [&](bool special, int gr, int key0, uint32_t bad) {
      // operands come from LDS a window ahead of the products (left alone, the compiler reads
      // one, waits, and multiplies: 16-token trees 18.0 us against 17.0)
      // (where registers are short, one at a time, in pairs of products)
      constexpr int WIN = 4, KN = 2 * G::KS;
      constexpr bool AHEAD = D * WGS < 256;
      uint4 win[AHEAD ? WIN : 1];
      auto k_at = [&](int n) { return sk(gr, n & 1, n >> 1); };
      v4f s[1][2] = {{v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}}};
      if constexpr (AHEAD) {
#pragma unroll
        for (int n = 0; n < WIN; ++n) win[n] = k_at(n);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int n = 0; n < KN; ++n) {
        s[0][n & 1] = mfma_bf16_16x16x32(AHEAD ? win[n % WIN] : k_at(n), q[n >> 1], s[0][n & 1]);
        if constexpr (AHEAD) win[n % WIN] = n + WIN < KN ? k_at(n + WIN) : sv(gr, n + WIN - KN);  // then the values' first
        if (AHEAD || (n & 1)) __builtin_amdgcn_sched_barrier(0);
      }
      uint4 pb[1];
      uint32_t vis[1] = {0};
      if (special) {
        vis[0] = (bad >> (g >> 1)) & 1u ? 0u : visible8(p, smask, sq.q0, min((row0 + i) / p.group, sq.n - 1), key0 + 8 * g - prefix, sq.n);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0][e >> 2][e & 3] = (vis[0] >> e) & 1u ? s[0][e >> 2][e & 3] : NEG_INF;
      }
      softmax_step<NT, 1, false>(s, sc, vis, m, l, o, pb);
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) {
        o[0][tt] = mfma_bf16_16x16x32(AHEAD ? win[(KN + tt) % WIN] : sv(gr, tt), pb[0], o[0][tt]);
        if constexpr (AHEAD)
          if (tt + WIN < NT) win[(KN + tt) % WIN] = sv(gr, tt + WIN);
        if (AHEAD || (tt & 1)) __builtin_amdgcn_sched_barrier(0);
      }
      if (special) {
#pragma unroll
        for (int part = 0; part < PARTS / 2; ++part) {
          const uint32_t odd = __builtin_amdgcn_readfirstlane((int)s_odd[gr][part]);
          if (odd) {
            auto at = [&](int key) {
              const int id = ld_table(table + (key >> p.page_log2));  // a page that exists: its keys are seen
              return reinterpret_cast<const char*>(p.v_cache) + ((((long)id * p.n_kv + h) << p.page_log2) + (key & (page - 1))) * G::ROWB;
            };
            add_odd_keys<D, FP8, PARTS / 2>(odd, odd & 0xffffu ? at(key0) : nullptr, odd >> 16 ? at(key0 + 16) : nullptr, pb[0], vis[0], o[0], part);
          }
        }
      }
    };

    for (int t = g0; t < g1; t += GR) {
      __syncthreads();  // the round before is read, and its masks, which may be another sequence's
      if (t == g0 && tid < 64) smask[tid] = mask_row;
      stage(t);
      if (t + GR < g1) fetch(t + GR);
      __syncthreads();
      for (int gr = mine_of; gr < GR && t + gr < g1 && busy; gr += split) {
        const int key0 = (t + gr) * ATTN_GROUP;
        const uint32_t bad = __builtin_amdgcn_readfirstlane((int)s_bad[gr]);
        group(key0 + 32 > prefix || bad, gr, key0, bad);
      }
    }

    l[0] += __shfl_xor(l[0], 16);
    l[0] += __shfl_xor(l[0], 32);
    if (split > 1) {  // join the waves of a tile, in order, in the first of them
      v4f* so = reinterpret_cast<v4f*>(ops);
      __syncthreads();  // the last round is read
      if (mine_of) {
        const int at = (wave - tiles) * NT;
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) so[(at + tt) * 64 + lane] = o[0][tt];
        if (g == 0) sml[wave][i] = make_float2(m[0], l[0]);
      }
      __syncthreads();
      if (mine_of == 0) {
        for (int w = 1; w < split; ++w) {
          const float2 ml = sml[tile + w * tiles][i];
          const float mn = fmaxf(m[0], ml.x);
          const float f = m[0] == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(m[0] - mn);
          const float fw = ml.x == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(ml.x - mn);
          const int at = (tile + (w - 1) * tiles) * NT;
          m[0] = mn;
          l[0] = l[0] * f + ml.y * fw;
#pragma unroll
          for (int tt = 0; tt < NT; ++tt) o[0][tt] = o[0][tt] * f + so[(at + tt) * 64 + lane] * fw;
        }
      }
    }
    if (busy && mine_of == 0) {
      if (whole) {
        put_tile<D, G::CH>(p, sq.q0, rows, h, row0 + i, g, o[0], m[0], l[0], FP8 ? p.v_scale[h] : 1.f);
      } else {
        float* dst = p.part_o + ((long)slot * (BLOCK / 16) + tile) * (16 * D) + 4 * lane;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int t4 = 0; t4 < NT; t4 += 4)
            *reinterpret_cast<float4*>(dst + (x * (NT / 4) + t4 / 4) * 256) =
                make_float4(o[0][t4][x], o[0][t4 + 1][x], o[0][t4 + 2][x], o[0][t4 + 3][x]);
        if (g == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * ((long)slot * BLOCK + tile * 16 + i)) = make_float2(m[0], l[0]);
      }
    }
  }
}

// Joins the pieces of k_tree_attention_rows: a workgroup a row tile, a wave one x of it.  The
// pieces are taken KR at a time with a running maximum, so that all loads of a round, the
// pieces' (m, l) among them, are in flight together: the launch is a chain of latencies (a
// pass of its own over the maxima, and a wave for a whole tile, took 10.8 us at 64 rows; this 6.3,
// and 9.3 for 248 units of up to 128 rows, whose pieces are 20 MB written and read).
template <int D, int CH>
__global__ __launch_bounds__(256) void k_tree_combine_rows(TreeAttnParams p, int block_rows) {
  constexpr int NV = D / 64, KR = D == 256 ? 4 : 8;  // float4 of a lane; pieces of a round
  const int wg = blockIdx.x, tile = blockIdx.y;
  const int4 ds = *reinterpret_cast<const int4*>(p.desc + ATTN_DESC * wg);
  const int rb = p.desc[ATTN_DESC * wg + 4];
  if (ds.x == 0) return;
  const int lane = threadIdx.x & 63, x = threadIdx.x >> 6, g = lane >> 4;
  const int rows = ds.z, r = rb * block_rows + tile * 16 + (lane & 15);
  if (r - (lane & 15) >= rows) return;
  const float* ml = p.part_ml + 2 * (tile * 16 + (lane & 15));
  const float* src = p.part_o + (long)tile * (16 * D) + x * NV * 256 + 4 * lane;
  float M = NEG_INF, L = 0.f;
  float4 o[NV];
#pragma unroll
  for (int t = 0; t < NV; ++t) o[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < ds.x; k0 += KR) {
    float2 v[KR];
    float4 u[KR][NV];
#pragma unroll
    for (int k = 0; k < KR; ++k) {
      const int kk = min(k0 + k, ds.x - 1);  // the last piece again, with no weight
      const long slot = kk == 0 ? 2 * wg + 1 : 2 * (wg + kk);
      v[k] = *reinterpret_cast<const float2*>(ml + 2 * slot * block_rows);
#pragma unroll
      for (int t = 0; t < NV; ++t) u[k][t] = *reinterpret_cast<const float4*>(src + slot * block_rows * D + t * 256);
    }
    float mn = M;
#pragma unroll
    for (int k = 0; k < KR; ++k) mn = fmaxf(mn, v[k].x);
    const float back = M == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(M - mn);
    L *= back;
#pragma unroll
    for (int t = 0; t < NV; ++t) { o[t].x *= back; o[t].y *= back; o[t].z *= back; o[t].w *= back; }
    M = mn;
#pragma unroll
    for (int k = 0; k < KR; ++k) {
      // selected, not branched around: a branch would pull the loads apart, one wait each
      const bool real = k0 + k < ds.x;
      const float f = v[k].x == NEG_INF ? 0.f : __builtin_amdgcn_exp2f(v[k].x - M);
      L += real ? v[k].y * f : 0.f;
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        o[t].x += real ? u[k][t].x * f : 0.f; o[t].y += real ? u[k][t].y * f : 0.f;
        o[t].z += real ? u[k][t].z * f : 0.f; o[t].w += real ? u[k][t].w * f : 0.f;
      }
    }
  }
  if (r >= rows) return;
  const float inv = L == 0.f ? 0.f : (p.v_scale ? p.v_scale[ds.w] : 1.f) / L;
  const int j = r / p.group;
  const long at = (long)(ds.y + j) * p.n_q + ds.w * p.group + (r - j * p.group);
#pragma unroll
  for (int t = 0; t < NV; ++t)  // tiles 4 t .. 4 t + 3: chunk 4 t / CH, places e = 4 t % CH ..
    *reinterpret_cast<uint2*>(p.out + at * D + 16 * CH * (4 * t / CH) + CH * (4 * g + x) + 4 * t % CH) =
        make_uint2(bf16x2_rne(o[t].x * inv, o[t].y * inv), bf16x2_rne(o[t].z * inv, o[t].w * inv));
  if (g == 0 && x == 0 && p.lse) p.lse[at] = L == 0.f ? NEG_INF : (M + __builtin_amdgcn_logf(L)) * 0.69314718055994531f;
}

// Bit i of row t: drafted token i is t or one of its ancestors.  A workgroup takes a sequence and
// a word of its masks, in LDS: mask(t) starts as t's own bit and up(t) as its parent; each round
// sets mask(t) |= mask(up(t)), up(t) = up(up(t)), so that k rounds reach 2^k ancestors.  A chain
// of latencies either way: following parents one by one through memory took 12.4 us for 16 chains
// of 64 and 136 us for 16 of 512, this 4.2 and 7.3.
constexpr int MASK_MOST = 1024;  // tokens of a sequence: 64 bits a word, 16 words at most
__global__ __launch_bounds__(256) void k_tree_mask(const int* parents, const int* q_indptr, int B, int T, int max_q,
                                                   int words, uint64_t* mask, int* status) {
  __shared__ uint64_t bits[2][MASK_MOST];
  __shared__ short up[2][MASK_MOST];
  const int b = blockIdx.x, w = blockIdx.y, q0 = q_indptr[b], q1 = q_indptr[b + 1];
  auto clear = [&](int from, int to) {  // rows that no sequence has: of these, where offsets descend,
    int back = 0;                       // those that no other sequence has
    for (int o = threadIdx.x; o < B; o += 256) back |= q_indptr[o + 1] < q_indptr[o];
    back = __syncthreads_or(back);
    for (int t = max(from, 0) + (int)threadIdx.x; t < min(to, T); t += 256) {
      bool taken = false;
      for (int o = 0; back && o < B && !taken; ++o) {
        const int o0 = q_indptr[o], o1 = q_indptr[o + 1];
        taken = tokens_fit(o0, o1, T, max_q) && o0 <= t && t < o1;
      }
      if (!taken) mask[(long)t * words + w] = 0;
    }
    if (threadIdx.x == 0 && status) or_agent(status, ST_LENGTH);
  };
  if (b == 0 && q0 > 0) clear(0, q0);
  if (b == B - 1 && q1 < T) clear(q1, T);
  if (q0 < 0 || q1 < q0 || q1 > T || q1 - q0 > max_q) {
    clear(q0, q1);
    return;
  }
  const int n = q1 - q0;
  for (int j = threadIdx.x; j < n; j += 256) {
    const int u = parents[q0 + j];
    if (u >= j && status) or_agent(status, ST_PARENT);
    bits[0][j] = j >> 6 == w ? 1ull << (j & 63) : 0ull;
    up[0][j] = (short)(u < j ? max(u, -1) : -1);
  }
  __syncthreads();
  int now = 0;
  for (int more = 1; more;) {  // ends: every up(t) is below t, or -1
    more = 0;
    for (int j = threadIdx.x; j < n; j += 256) {
      const int u = up[now][j];
      uint64_t m = bits[now][j];
      int next = -1;
      if (u >= 0) {
        m |= bits[now][u];
        next = up[now][u];
      }
      bits[now ^ 1][j] = m;
      up[now ^ 1][j] = (short)next;
      more |= next >= 0;
    }
    more = __syncthreads_or(more);
    now ^= 1;
  }
  for (int j = threadIdx.x; j < n; j += 256) mask[(long)(q0 + j) * words + w] = bits[now][j];
}

template <int D, int RT, bool FP8>
void launch_few(const TreeAttnParams& p, hipStream_t s) {
  constexpr int OCC = RT == 1 && D <= 128 ? 2 : 1;
  hipLaunchKernelGGL((k_tree_attention<D, RT, FP8, OCC>), dim3(p.n_wg), dim3(256), (p.B + 1) * sizeof(int), s, p);
  const int rows = min(RT * 16, p.max_q * p.group);
  // a workgroup a row where few units are cut into many pieces (64 pieces of 4 rows: 5.9 us
  // against 9.0; 4 pieces of 4 rows 5.6 against 4.0)
  if (rows <= 4 && p.B * p.n_kv * 16 <= p.n_wg)
    hipLaunchKernelGGL((k_tree_combine<D, true>), dim3(p.n_wg, rows), dim3(256), 0, s, p, RT * 16);
  else
    hipLaunchKernelGGL((k_tree_combine<D, false>), dim3(p.n_wg, (rows + 3) / 4), dim3(256), 0, s, p, RT * 16);
}

template <int D, bool FP8, int WGS>
void launch_rows(const TreeAttnParams& p, hipStream_t s) {
  constexpr int BLOCK = 16 * ROW_WAVES;
  hipLaunchKernelGGL((k_tree_attention_rows<D, FP8, WGS>), dim3(p.n_wg), dim3(64 * ROW_WAVES), (p.B + 1) * sizeof(int), s, p);
  const long rows = min((long)BLOCK, (long)p.max_q * p.group);
  hipLaunchKernelGGL((k_tree_combine_rows<D, Geo<D, FP8>::CH>), dim3(p.n_wg, (unsigned)((rows + 15) / 16)), dim3(256), 0, s, p, BLOCK);
}

template <int D, bool FP8>
hipError_t launch_d(const TreeAttnParams& p, const TreeAttnPlan& pl, hipStream_t s) {
  if (pl.shared) {
    if constexpr (D <= 128) {
      if (pl.n_wg > 256) launch_rows<D, FP8, 2>(p, s);
      else launch_rows<D, FP8, 1>(p, s);
    } else {
      launch_rows<D, FP8, 1>(p, s);
    }
  } else {
    if (pl.row_tiles == 1) launch_few<D, 1, FP8>(p, s);
    else if constexpr (D <= 128 && FP8) launch_few<D, 2, FP8>(p, s);
  }
  return hipGetLastError();
}

}  // namespace

TreeAttnPlan tree_attn_plan(int D, int max_q, int group, bool fp8, bool mask, long heads) {
  const long rows = (long)max_q * group;
  TreeAttnPlan pl;
  pl.counted = false;
  // 17 to 32 rows of an 8-bit cache: waves that split the keys, with two tiles of rows (heads of
  // 256: two blocks), do not put what they widen through LDS (32 sequences of 2,048 keys, 32 rows:
  // 40 us against 48, heads of 256 99 against 112; in 16 bits 58 against 55 and 189 against 108)
  pl.shared = rows > (fp8 ? 32 : 16);
  if (pl.shared) {
    pl.row_tiles = 1;
    pl.block_rows = 16 * ROW_WAVES;
    const long units = heads * ((rows + pl.block_rows - 1) / pl.block_rows);
    // two workgroups a CU from 512 units on (heads of 64: 384), where they are not cut into twice
    // the pieces. Sequences of 2,048 keys, 8 kv heads, one and two a CU, in us: heads of 128, 8-bit
    // cache, 64 sequences of 64 rows 108 and 91, 32 of 256 rows 130 and 115, 48 of 64 (384 units)
    // 88 and 85; 16-bit 64 of 128 rows 147 and 133, 48 of 64 95 and 105; heads of 64, 64 of 64
    // rows 73 and 50, 48 of 64 55 and 47, 32 of 128 (256 units) 46 and 53
    pl.n_wg = D <= 128 && units >= (D == 64 ? 384 : 512) ? 512 : 256;
    // A prompt's row blocks count what they see (32 + 8 + 8 heads of 128, in us, all alike and so:
    // prompts of 1,024 tokens, 4 of them, 147 and 120, of 4,096 465 and 304, of 700, 4, 96 and 75, of
    // 256, 32, 83 and 71; 800 more tokens of 8,000 178 and 170).  Not where all alike gives almost
    // every workgroup a unit of its own and cuts none (8 prompts of 256 30 and 43, 512 more tokens of
    // 2,048, 4, 113 and 126), unless the prompts are long (2,048: 126 and 110).  Units go by max_q, the
    // one length that the host has.  In us, all alike and counted: 4 prompts of 256 19 and 30, on 2,000
    // tokens each 67 and 81, two of 512 27 and 37, on 8,000 205 and 218; where the lengths are ragged the
    // units are fewer and are cut all the same: 256, 100, 250 and 180 tokens 29 and 26, eight of 30 to
    // 256 34 and 33, one of 256 beside three decoding sequences 39 and 38.  (Heads of 64 and 8-bit caches
    // alike.)
    const bool own = units <= pl.n_wg && 8 * units > 7 * pl.n_wg && max_q < 1024;
    pl.counted = !mask && rows > pl.block_rows && !own;
  } else {
    pl.row_tiles = rows <= 16 || D > 128 ? 1 : 2;
    pl.block_rows = 16 * pl.row_tiles;
    pl.n_wg = pl.row_tiles == 1 && D <= 128 ? 512 : 256;  // what the registers let run at once: two a CU, or one
  }
  const size_t slots = 2 * (size_t)pl.n_wg, r = (size_t)pl.block_rows;
  pl.desc_bytes = (size_t)pl.n_wg * ATTN_DESC * 4;
  pl.ml_bytes = slots * r * 8;
  pl.o_bytes = slots * r * D * 4;
  return pl;
}

hipError_t launch_tree_attention(const TreeAttnParams& p, const TreeAttnPlan& pl, int D, bool fp8, hipStream_t s) {
  switch (D) {
    case 64: return fp8 ? launch_d<64, true>(p, pl, s) : launch_d<64, false>(p, pl, s);
    case 128: return fp8 ? launch_d<128, true>(p, pl, s) : launch_d<128, false>(p, pl, s);
    default: return fp8 ? launch_d<256, true>(p, pl, s) : launch_d<256, false>(p, pl, s);
  }
}

hipError_t launch_tree_mask(const int* parents, const int* q_indptr, int B, int T, int max_q, int words, uint64_t* mask,
                            int* status, hipStream_t s) {
  hipLaunchKernelGGL(k_tree_mask, dim3(B, words), dim3(256), 0, s, parents, q_indptr, B, T, max_q, words, mask, status);
  return hipGetLastError();
}

}  // namespace lora
