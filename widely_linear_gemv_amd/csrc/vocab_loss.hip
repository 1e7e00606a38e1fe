// Softmax cross entropy over a large vocabulary without keeping the logits, and its gradient.
//
//     l_iv = <h_i, W_v>,  lse_i = log sum_v exp l_iv,  loss_i = lse_i - l_{i, t_i}
//     p_iv = g_i (exp(l_iv - lse_i) - [v = t_i]),  dh_i = sum_v p_iv W_v,  dW_v = sum_i p_iv h_i
//
// One tiled product C = A B^T (rows of A and B contiguous along the contraction) on the matrix
// cores does all the work; what differs is what happens to a finished tile:
//   logits   A = W, B = h: each tile is reduced on chip to a (maximum, sum of exponentials) pair
//            per token, and the target's logit is picked out; no logit is stored.
//   p        the same product again for a piece of the vocabulary: p [token][v] is rounded to the
//            inputs' dtype and stored.
//   dh       A = W^T, B = p: fp32 sums over the pieces, rounded once at the end.
//   dW       A = h^T, B = p^T: rows of the piece, rounded once.
// For bf16 inputs the rounding of p (2^-8) must not move whole rows: the entry -g_i (1 - p_t) of a token's
// target t dominates dh_i and row t of dW, so its rounding would be all of a row's values' at once (and,
// where all g are equal, every row's).  So p is stored in units in which that entry is a power of two: with
// f_i = 1 - softmax_t, g_i f_i is taken apart as G m_i s_i with 1 <= G < 2 the significand of the first
// token's |g|, s_i a power of two with g_i's sign and 1/2 < m_i <= 1; p holds -s_i for the target and
// s_i softmax / f_i elsewhere, dh_i is scaled by G m_i and dW by G in fp32, and dW's other operand is m_i h_i
// (h itself to within f_i where all g are equal, as for a mean).  Then the roundings, of p's other entries
// and of m_i h_i, are independent from value to value.  Target probabilities of 0.2 to 0.7, 256 tokens, 2000 x
// 1024: dh 0.00166 off 64 bits (2-norm), as much as its own final rounding; dW 0.0024, final rounding 0.0017.
// (Where f_i is under 2^-16, mostly rounding itself, it is left in p: the target's entry is then
// -s_i (1 - softmax_t).)
// No part leaves fp32's range: p and the sums keep g's own size to within a factor of 4, but for |g_i| f_i
// under 2^-60, where s_i stays at 2^-60 (or p would lose its small values) and m_i takes the rest.
// Transposed operands are read from the matrix as it lies in memory: rows of the contraction are
// copied into LDS and transposed on the way into registers, so no transposed copy is made.
// Sums are fp32; a C tile has the A rows in its accumulator rows, so a lane holds four consecutive
// vocabulary entries (or hidden columns) of one token (or vocabulary row).
#include <algorithm>

#include "tiles.hpp"

namespace f2i {

namespace {

enum { kLoss = 0, kGrad = 1, kHidden = 2, kWeight = 3 };

// acc += a b on the matrix cores, one 16-byte operand per lane.  The accumulator is tied to its own
// accumulation registers: left to itself the compiler moves the 256 of a 128 x 128 wave tile about,
// which cost a third of the time.  (Consecutive calls use different accumulators, and settle()
// separates the last one from whatever reads them.)
__device__ __forceinline__ void mma(v4f& acc, const v4u& a, const v4u& b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// exp(x) for x <= 0: off by 1.25 |x| 2^-24 of itself (the product's rounding, and the constant's, a quarter
// of that) and by the exp2 instruction's own error, about a unit in the last place (2^-23).  In
// sum_v exp(l_v - top) that comes to at most 1.25 log(V) 2^-24 + 2^-23 of the sum (the mean distance from the
// maximum under the softmax is at most log V).
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// exp(l - top), 1 where both are the same infinity.
__device__ __forceinline__ float exp_off(float l, float top) { return l == top ? 1.f : fast_exp(l - top); }

}  // namespace

// What the epilogues need.
struct VocabTile {
  int64_t rows_a, rows_b;       // rows of A and B
  int64_t k;                    // contraction
  int64_t lda, ldb;             // row pitch in memory (of a transposed operand: of its contraction rows)
  const void* a;
  const void* b;
  const int64_t* target;        // [N]
  const float* lse;             // [N] (kGrad; bf16: with log f_i added)
  const float* g;               // [N] factor of p (kGrad; bf16: s_i)
  const float* at_target;       // [N] p over that factor at the target (kGrad, bf16)
  const float* row_scale;       // [N] factor of dh's rows, or null (kHidden)
  const float* all_scale;       // [1] factor of dW, or null (kWeight)
  float2* part;                 // [row tile of A][N] (kLoss)
  float* tlogit;                // [N] (kLoss)
  void* p;                      // [N][ldp] (kGrad)
  float* acc;                   // [splits][rows_b][rows_a] fp32 running sums (kHidden)
  void* out;                    // [rows_b][rows_a] (kHidden on the last piece, kWeight)
  int64_t v0, V;                // first vocabulary entry of A, vocabulary size
  int64_t N, ldp;
  int first, last;              // piece
  int tiles_a, tiles_b;
  int splits;                   // of the contraction (kHidden; 1 otherwise)
};

// What happens to a finished tile (above).
template <typename T, int BM, int BN, int WA, int WB, int FA, int FB, int EPI>
__device__ __forceinline__ void finish(const VocabTile& t, v4f (&acc)[FA][FB], uint8_t* s_buf, int64_t a0, int64_t b0,
                                       int ta, int split) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int wa = wave / WB, wb = wave % WB;
  const int64_t va = a0 + wa * FA * 16 + 4 * g;            // this lane's first A row
  const int64_t nb = b0 + wb * FB * 16 + c;                // its first B row
  if constexpr (EPI == kLoss) {
    // The pairs of the tile's waves take over the operand buffers.  (They are not an array of their own:
    // with two arrays in LDS the compiler no longer knows that an operand read cannot meet a copy in
    // flight and waits for every copy before every read, which doubled the time.)
    __syncthreads();                                       // every wave's copies have landed
    float2(*s_red)[BN] = reinterpret_cast<float2(*)[BN]>(s_buf);
    static_assert(WA * BN * sizeof(float2) <= (BM + BN) * 128, "the pairs fit");
    const bool whole = a0 + BM <= t.V;                     // no row past the vocabulary
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int64_t tok = nb + 16 * j;
      const int64_t tgt = tok < t.N ? t.target[tok] : -1;
      // this lane has the target's logit if it lies 16 i + e past the lane's first row
      const int d = tgt >= va && tgt < va + FA * 16 && tgt < t.V ? (int)(tgt - va) : 4;
      float top = -INFINITY, mine = 0.f;
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!whole && va + 16 * i + e >= t.V) acc[i][j][e] = -INFINITY;
          top = fmaxf(top, acc[i][j][e]);
        }
      if (__ballot((d & 12) == 0)) {
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (d == 16 * i + e) mine = acc[i][j][e];
        if ((d & 12) == 0) t.tlogit[tok] = mine;
      }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      float sum = 0.f;
      if (__ballot(!(fabsf(top) < INFINITY))) {            // an infinity: exp_off's cases
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (va + 16 * i + e < t.V) sum += exp_off(acc[i][j][e], top);
      } else {
#pragma unroll
        for (int i = 0; i < FA; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += fast_exp(acc[i][j][e] - top);
      }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0) s_red[wa][(wb * FB + j) * 16 + c] = make_float2(top, sum);
    }
    __syncthreads();
    for (int k = tid; k < BN; k += 64 * WA * WB) {
      if (b0 + k >= t.N) continue;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WA; ++w) top = fmaxf(top, s_red[w][k].x);
#pragma unroll
      for (int w = 0; w < WA; ++w) sum += s_red[w][k].y * exp_off(s_red[w][k].x, top);
      t.part[(int64_t)ta * t.N + b0 + k] = make_float2(top, sum);
    }
  } else if constexpr (EPI == kGrad) {
    T* __restrict__ p = static_cast<T*>(t.p);
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int64_t tok = nb + 16 * j;
      if (tok >= t.N) continue;
      const int64_t tgt = t.target[tok];
      const float gi = tgt >= 0 && tgt < t.V ? t.g[tok] : 0.f;
      const bool live = gi != 0.f;                         // other tokens give 0 whatever their logits are
      const float lse = live ? t.lse[tok] : 0.f;
      float at_target = 0.f;
      if constexpr (sizeof(T) == 2) at_target = live ? t.at_target[tok] : 0.f;
      const int64_t away = tgt - t.v0 - va;                // the target lies this far past the lane's first row
      const int d = live && away >= 0 && away < FA * 16 ? (int)away : -1;
#pragma unroll
      for (int i = 0; i < FA; ++i) {
        const int64_t r = va + 16 * i;                     // row within the piece
        if (r >= t.ldp) continue;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool target = d == 16 * i + e;
          float v;
          if constexpr (sizeof(T) == 2) v = target ? at_target : fast_exp(acc[i][j][e] - lse);
          else v = expf(acc[i][j][e] - lse) - (target ? 1.f : 0.f);
          x[e] = live && r + e < t.rows_a ? gi * v : 0.f;
        }
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(p + tok * t.ldp + r) =
              make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        else
          *reinterpret_cast<v4f*>(p + tok * t.ldp + r) = v4f{x[0], x[1], x[2], x[3]};
      }
    }
  } else {
    T* __restrict__ out = static_cast<T*>(t.out);
    const float all = EPI == kWeight && t.all_scale ? *t.all_scale : 1.f;
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int64_t rowb = nb + 16 * j;
      if (rowb >= t.rows_b) continue;
      const float scale = EPI == kHidden && t.row_scale ? t.row_scale[rowb] : all;
#pragma unroll
      for (int i = 0; i < FA; ++i) {
        const int64_t col = va + 16 * i;
        if (col >= t.rows_a) continue;                     // rows_a is a multiple of 64
        const int64_t at = rowb * t.rows_a + col;
        v4f v = acc[i][j];
        if constexpr (EPI == kHidden) {
          float* sum = t.acc + (int64_t)split * t.rows_b * t.rows_a + at;
          if (!t.first) v += *reinterpret_cast<const v4f*>(sum);
          if (!t.last || t.splits > 1) {
            *reinterpret_cast<v4f*>(sum) = v;
            continue;
          }
        }
        v *= scale;
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(out + at) =
              make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else
          *reinterpret_cast<v4f*>(out + at) = v;
      }
    }
  }
}

// Workgroup: a BM x BN tile of C, WA x WB waves, each BM/WA x BN/WB.  The contraction runs in steps of
// 128 bytes (64 values) of every row -- whole cache lines: 64-byte pieces halved the L2's throughput --
// in NB buffers in LDS (two; four where one workgroup a CU streams W past few tokens and needs the bytes
// in flight), each step multiplied in two halves.  While a half is multiplied
// (its operands already in registers) the wave reads the next half's operands from LDS; once a step's
// second half is in registers everywhere (the step's one barrier), the copies of step s + NB go straight
// into its buffer and have NB - 1.5 steps to land.  Rows
// past the end of a matrix read as 0; past the last step the copies repeat it, which nothing reads.
//
// Bound by the matrix cores under the power limit for many tokens: 2048 x 32000 x 4096 takes 400-500 us as
// logits (1342-1074 TFLOP/s; the card's best library product reaches 1399 at 8192^3; on zeros the same
// launch takes 365), 431-451 as p, 460-491 as dh and 464-507 as dW.  For 24 tokens by W from HBM:
// 262 MB in 59 us, 4.4 TB/s (two buffers 64 us).
template <int BM, int BN, int WA, int WB, int EPI, int NB = 2>
__global__ __launch_bounds__(64 * WA * WB, 1) void k_nt(VocabTile t) {
  using T = uint16_t;
  constexpr int kWaves = WA * WB;
  constexpr int FA = BM / WA / 16, FB = BN / WB / 16;
  constexpr int kBlocks = (BM + BN) / 8;                  // 1 KB copies per step
  static_assert(BM / 8 % kWaves == 0 && BN / 8 % kWaves == 0, "whole copies per wave and side");
  constexpr int kMine = kBlocks / kWaves;
  constexpr int kStep = (BM + BN) * 128;
  constexpr int kDeep = 128 / sizeof(T);                  // contraction per step
  using SideA = Side<T, BM, (EPI == kHidden || EPI == kWeight)>;
  using SideB = Side<T, BN, EPI == kWeight>;
  constexpr bool kTransA = EPI == kHidden || EPI == kWeight, kTransB = EPI == kWeight;
  // waits until at most `steps` steps' copies of this wave are in flight (and for its LDS reads: lgkm 0)
  constexpr auto wait = [](int steps, int lgkm) {
    return (steps * kMine & 15) | ((steps * kMine >> 4) << 14) | 0x70 | (lgkm << 8);
  };
  static_assert((NB - 1) * kMine < 64 && (NB & (NB - 1)) == 0, "the copies in flight can be counted");
  __shared__ __align__(16) uint8_t s_buf[NB * kStep];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int wa = wave / WB, wb = wave % WB;
  // Workgroups go to the eight XCDs in turn; each XCD takes a contiguous run of tiles with the B tiles
  // innermost, so the A rows of a run are fetched into one L2 only.
  const int split = blockIdx.y;
  const int per_xcd = (t.tiles_a * t.tiles_b + 7) / 8;
  const int tile = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || tile >= t.tiles_a * t.tiles_b) return;
  const int ta = tile / t.tiles_b, tb = tile % t.tiles_b;
  const int64_t a0 = (int64_t)ta * BM, b0 = (int64_t)tb * BN;
  const int all_steps = (int)((t.k + kDeep - 1) / kDeep);
  const int per_split = (all_steps + t.splits - 1) / t.splits;
  const int step0 = split * per_split, steps = min(per_split, all_steps - step0);
  // the part of an operand that step `step` copies, and the lanes' offsets in it
  auto part = [&](const void* m, int64_t row0, int64_t rows, int64_t ld, bool trans, int step) {
    const T* p = static_cast<const T*>(m);
    if (trans) {
      const int64_t k = (int64_t)step * kDeep;
      return range_rsrc(p + k * ld, max(t.k - k, (int64_t)0) * ld * (int64_t)sizeof(T));
    }
    return range_rsrc(p + row0 * ld, max(rows - row0, (int64_t)0) * ld * (int64_t)sizeof(T));
  };
  // Copy i of this wave is 1 KB number i kWaves + wave of the step; the first kCopiesA are A's.
  constexpr int kCopiesA = BM / 8 / kWaves;
  uint32_t off[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int blk = i * kWaves + wave;
    off[i] = i < kCopiesA ? SideA::source(blk, lane, t.lda) + (kTransA ? (uint32_t)(a0 * sizeof(T)) : 0)
                          : SideB::source(blk - BM / 8, lane, t.ldb) + (kTransB ? (uint32_t)(b0 * sizeof(T)) : 0);
  }
  auto copy = [&](__amdgpu_buffer_rsrc_t rs_a, __amdgpu_buffer_rsrc_t rs_b, int step, int buf, int from, int to) {
    const int ka = kTransA ? 0 : step * 128, kb = kTransB ? 0 : step * 128;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (i < from || i >= to) continue;
      const uint32_t voff = off[i];
      uint8_t* to_lds = s_buf + buf * kStep + (i * kWaves + wave) * 1024;
      if (i < kCopiesA) __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, (lds_ptr_t)to_lds, 16, voff, ka, 0, 0);
      else __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, (lds_ptr_t)to_lds, 16, voff, kb, 0, 0);
    }
  };
  v4f acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  if (steps > 0) {
    v4u fa[2][FA], fb[2][FB];
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      const int step = step0 + min(r, steps - 1);
      copy(part(t.a, a0, t.rows_a, t.lda, kTransA, step), part(t.b, b0, t.rows_b, t.ldb, kTransB, step), step, r, 0, kMine);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait(NB - 1, 15));          // step 0 has landed
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < FA; ++i) fa[0][i] = SideA::read(s_buf, wa * FA + i, 0, c, g);
#pragma unroll
    for (int j = 0; j < FB; ++j) fb[0][j] = SideB::read(s_buf + BM * 128, wb * FB + j, 0, c, g);
    for (int s = 0; s < steps; ++s) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // FA groups of FB products; ahead of each group its share of the reads and copies
        const uint8_t* next = s_buf + ((s + h) & (NB - 1)) * kStep;
        const int after = step0 + min(s + NB, steps - 1);
        const __amdgpu_buffer_rsrc_t rs_a = part(t.a, a0, t.rows_a, t.lda, kTransA, after);
        const __amdgpu_buffer_rsrc_t rs_b = part(t.b, b0, t.rows_b, t.ldb, kTransB, after);
#pragma unroll
        for (int i = 0; i < FA; ++i) {
          fa[h ^ 1][i] = SideA::read(next, wa * FA + i, h ^ 1, c, g);
#pragma unroll
          for (int j = i * FB / FA; j < (i + 1) * FB / FA; ++j)
            fb[h ^ 1][j] = SideB::read(next + BM * 128, wb * FB + j, h ^ 1, c, g);
          if (h == 1) copy(rs_a, rs_b, after, s & (NB - 1), i * kMine / FA, (i + 1) * kMine / FA);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < FB; ++j) mma(acc[i][j], fa[h][i], fb[h][j]);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (h == 0) {
          // this wave holds the step's second half, and its copies of the next step have landed
          asm volatile("" ::: "memory");
          __builtin_amdgcn_s_waitcnt(wait(NB - 2, 0));
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0);                         // no copy outlives its buffer
    settle();
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) asm volatile("" : "+a"(acc[i][j]));   // read only after settle()
  }

  finish<T, BM, BN, WA, WB, FA, FB, EPI>(t, acc, s_buf, a0, b0, ta, split);
}

// The same product for fp32 operands, on the bf16 matrix instructions: every value is cut into three bf16
// parts of 8 bits each (x = x1 + x2 + x3 exactly: each part is what is left, rounded to nearest, so
// |x2| <= 2^-8 and |x3| <= 2^-17 of x's power of two), and of the nine products of two values' parts the six
// largest are summed; the other three are at most (1 + 2^-9) 2^-24 of |a b| together and of either sign,
// within the rounding of the fp32 sums.  (Parts cut off instead of rounded leave up to 2^-21, always of a b's
// own sign: every sum shrinks.)  Six bf16 products take 96 cycles of a SIMD for 16 x 16 x 32, the fp32
// instructions 256.
//
// Workgroup and waves as k_nt.  Steps of 32 along the contraction: while step s is multiplied from one of
// two LDS buffers, each thread cuts its 16-byte pieces of step s + 1 and writes the three parts to the
// other between the products, and then loads those of step s + 2 into the registers
// that this frees; one barrier a step.  (A second set of registers, loaded a step earlier, spilled: dW of
// 2048 x 32000 x 4096 3390 us against 3150.  Operands of the next step read between the products, or each
// piece's load issued right after its cut, changed nothing: 2228-2350 us either way.)
//
// Bound by the matrix cores under the power limit: 2048 x 32000 x 4096 takes 2.33-2.42 ms as logits, six
// bf16 products at 1383-1335 TFLOP/s (on zeros 2.08); p 2.38-2.46 ms, dh 2.42-2.48, dW 2.7.  263 x 5003 x
// 1088: 31-38 us each, 200 tiles of 128 x 64 on 256 CUs; a step takes 0.69 us, of which the products alone
// would be 0.32 and loads without anything else 0.32.  (With the parts cut off, two instructions fewer a pair:
// 0.66 us a step, without cuts 0.47, without loads 0.51.)
//   Plain operand: a part's row R is 64 bytes, its 16-byte segment sg in place sg ^ (R / 2 % 4).
//   Transposed: rows of the contraction as in Side<bf16, ROWS, true>.
template <int ROWS, bool TRANS, int THREADS>
struct SplitSide {
  static constexpr int kPart = ROWS * 64;                 // bytes of one part of a step
  static constexpr int kPieces = ROWS * 8 / THREADS;      // 16-byte pieces of a thread
  static_assert(ROWS * 8 % THREADS == 0, "whole pieces per thread");
  using Bf = Side<uint16_t, ROWS, true>;
  __device__ static uint32_t source(int i, int tid, int64_t ld) {
    const int u = i * THREADS + tid;
    if constexpr (TRANS) return (uint32_t)((u / (ROWS / 4)) * ld * 4) + (u % (ROWS / 4)) * 16;
    else return (uint32_t)((u / 8) * ld * 4) + (u % 8) * 16;
  }
  __device__ static int place(int i, int tid) {
    const int u = i * THREADS + tid;
    if constexpr (TRANS) {
      const int k = u / (ROWS / 4), q = u % (ROWS / 4);
      return k * ROWS * 2 + ((q >> 2) ^ Bf::f(k)) * 32 + (q & 3) * 8;
    } else {
      const int R = u / 8, q = u % 8;
      return R * 64 + ((q >> 1) ^ ((R >> 1) & 3)) * 16 + (q & 1) * 8;
    }
  }
  __device__ static __forceinline__ v4u read(const uint8_t* part, int frag, int c, int g) {
    if constexpr (TRANS) return Bf::read(part, frag, 0, c, g);
    else return *reinterpret_cast<const v4u*>(part + (frag * 16 + c) * 64 + ((g ^ ((c >> 1) & 3)) * 16));
  }
};

// Four fp32 values cut into parts, two bf16 to a word: out[p] holds part p.  The first part is at most the
// largest bf16, to which fp32 values past it would not round.  (Of an infinity NaN is left, so that its
// products are NaN.)
__device__ __forceinline__ void cut(const v4u& x, v2u (&out)[3]) {
  float f[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(x[e]);
#pragma unroll
  for (int p = 0; p < 3; ++p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      constexpr float kMost = 0x1.FEp127f;
      float a = f[2 * h], b = f[2 * h + 1];
      if (p == 0) {
        a = __builtin_amdgcn_fmed3f(a, -kMost, kMost);
        b = __builtin_amdgcn_fmed3f(b, -kMost, kMost);
      }
      out[p][h] = pack_bf16(a, b);
      f[2 * h] -= bf16_lo(out[p][h]);
      f[2 * h + 1] -= bf16_hi(out[p][h]);
    }
  }
}

template <int BM, int BN, int WA, int WB, int EPI>
__global__ __launch_bounds__(64 * WA * WB, 1) void k_nt_split(VocabTile t) {
  constexpr int kThreads = 64 * WA * WB;
  constexpr int FA = BM / WA / 16, FB = BN / WB / 16;
  constexpr bool kTransA = EPI == kHidden || EPI == kWeight, kTransB = EPI == kWeight;
  using SideA = SplitSide<BM, kTransA, kThreads>;
  using SideB = SplitSide<BN, kTransB, kThreads>;
  constexpr int kStep = 3 * (BM + BN) * 64;
  constexpr int PA = SideA::kPieces, PB = SideB::kPieces;
  __shared__ __align__(16) uint8_t s_buf[2 * kStep];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int wa = wave / WB, wb = wave % WB;
  const int split = blockIdx.y;
  const int per_xcd = (t.tiles_a * t.tiles_b + 7) / 8;    // as k_nt
  const int tile = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || tile >= t.tiles_a * t.tiles_b) return;
  const int ta = tile / t.tiles_b, tb = tile % t.tiles_b;
  const int64_t a0 = (int64_t)ta * BM, b0 = (int64_t)tb * BN;
  const int all_steps = (int)((t.k + 31) / 32);
  const int per_split = (all_steps + t.splits - 1) / t.splits;
  const int step0 = split * per_split, steps = min(per_split, all_steps - step0);
  auto part = [&](const void* m, int64_t row0, int64_t rows, int64_t ld, bool trans, int step) {
    const float* p = static_cast<const float*>(m);
    const int64_t from = trans ? (int64_t)step * 32 : row0, all = trans ? t.k : rows;
    return range_rsrc(p + from * ld, max(all - from, (int64_t)0) * ld * 4);
  };
  uint32_t off_a[PA], off_b[PB];
#pragma unroll
  for (int i = 0; i < PA; ++i) off_a[i] = SideA::source(i, tid, t.lda) + (kTransA ? (uint32_t)(a0 * 4) : 0);
#pragma unroll
  for (int i = 0; i < PB; ++i) off_b[i] = SideB::source(i, tid, t.ldb) + (kTransB ? (uint32_t)(b0 * 4) : 0);
  v4u raw_a[PA], raw_b[PB];
  auto load = [&](int step) {
    step = step0 + min(step, steps - 1);
    const __amdgpu_buffer_rsrc_t rs_a = part(t.a, a0, t.rows_a, t.lda, kTransA, step);
    const __amdgpu_buffer_rsrc_t rs_b = part(t.b, b0, t.rows_b, t.ldb, kTransB, step);
    const int ka = kTransA ? 0 : step * 128, kb = kTransB ? 0 : step * 128;
#pragma unroll
    for (int i = 0; i < PA; ++i) raw_a[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rs_a, off_a[i], ka, 0));
#pragma unroll
    for (int i = 0; i < PB; ++i) raw_b[i] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rs_b, off_b[i], kb, 0));
  };
  auto store = [&](int buf, int i) {                      // piece i of A, or i - PA of B
    uint8_t* base = s_buf + buf * kStep;
    v2u o[3];
    if (i < PA) {
      cut(raw_a[i < PA ? i : 0], o);
#pragma unroll
      for (int p = 0; p < 3; ++p) *reinterpret_cast<v2u*>(base + p * SideA::kPart + SideA::place(i, tid)) = o[p];
    } else {
      cut(raw_b[i < PA ? 0 : i - PA], o);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<v2u*>(base + 3 * SideA::kPart + p * SideB::kPart + SideB::place(i - PA, tid)) = o[p];
    }
  };
  v4f acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  if (steps > 0) {
    load(0);
#pragma unroll
    for (int i = 0; i < PA + PB; ++i) store(0, i);
    load(1);
    __syncthreads();
    for (int s0 = 0; s0 < steps; s0 += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int s = s0 + h;
        if (s >= steps) break;
        const uint8_t* from = s_buf + h * kStep;
        v4u fa[3][FA], fb[3][FB];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
#pragma unroll
          for (int i = 0; i < FA; ++i) fa[p][i] = SideA::read(from + p * SideA::kPart, wa * FA + i, c, g);
#pragma unroll
          for (int j = 0; j < FB; ++j) fb[p][j] = SideB::read(from + 3 * SideA::kPart + p * SideB::kPart, wb * FB + j, c, g);
        }
        // the six products, smallest parts first; the next step's pieces are cut between them
        constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
        for (int q = 0; q < 6; ++q) {
#pragma unroll
          for (int i = 0; i < FA; ++i)
#pragma unroll
            for (int j = 0; j < FB; ++j) mma(acc[i][j], fa[kA[q]][i], fb[kB[q]][j]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = q * (PA + PB) / 5; i < min(q + 1, 5) * (PA + PB) / 5; ++i) store(h ^ 1, i);
          if (q == 4) load(s + 2);
          __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
      }
    }
    settle();
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) asm volatile("" : "+a"(acc[i][j]));   // read only after settle()
  }
  finish<float, BM, BN, WA, WB, FA, FB, EPI>(t, acc, s_buf, a0, b0, ta, split);
}

// Joins the tiles' pairs in order (one wave per token) into lse, and the loss from the target's logit:
// launch-bound (4.6 us for 24 tokens, 5.2 for 2048).
__global__ __launch_bounds__(256) void k_loss_join(const float2* __restrict__ part, const float* __restrict__ tlogit,
                                                   const int64_t* __restrict__ target, int64_t N, int64_t V, int tiles,
                                                   float* __restrict__ loss, float* __restrict__ lse) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t i = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (i >= N) return;
  float top = -INFINITY;
  for (int s = lane; s < tiles; s += kWave) top = fmaxf(top, part[(int64_t)s * N + i].x);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  float sum = 0.f;
  for (int s = lane; s < tiles; s += kWave) {
    const float2 v = part[(int64_t)s * N + i];
    sum += v.y * exp_off(v.x, top);
  }
  sum = wave_sum(sum);
  if (lane == 0) {
    const float l = top + logf(sum);
    lse[i] = l;
    const int64_t t = target[i];
    loss[i] = t >= 0 && t < V ? l - tlogit[i] : 0.f;
  }
}

// out = the sum of the splits' running sums, in order, times the row's factor (if any), rounded once.
template <typename T>
__global__ __launch_bounds__(256) void k_hidden_join(const float* __restrict__ acc, const float* __restrict__ row_scale,
                                                     T* __restrict__ out, int64_t n, int64_t K, int splits) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;       // n and K are multiples of 64
  if (i >= n) return;
  v4f v = *reinterpret_cast<const v4f*>(acc + i);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const v4f*>(acc + s * n + i);
  if (row_scale) v *= row_scale[i / K];
#pragma unroll
  for (int e = 0; e < 4; ++e) store_out(out, i + e, v[e]);
}

// bf16: the parts of g f (above), one wave per token: s_i (0 for tokens that do not count or have g = 0),
// G m_i, p's target entry over s_i, lse_i + log f_i, and m_i h_i where `scaled` is given.  f_i comes from the
// target's logit, made here (off by as much as the product's own).  G is the significand of |g| of the first
// token that counts and has a finite g other than 0 (any number in [1, 2) would do; this one makes m_i 1 to
// within f_i where all g are equal); every wave finds it for itself, 64 tokens at a time, among the first 4096
// (with a longer run of padding in front G is 1: equal g then cost dW the rounding that different ones do).  A
// g that is not finite is its own s_i, so that it reaches its outputs.
// Rows of `scaled` are 0 for tokens that do not count or have g = 0: padding may hold anything, and p = 0
// times a NaN would be one in every row of dW.  fp32 needs the copy for this alone.  12-13 us for 2048 x 4096
// bf16 (8 without the target's logits), of a step's 1840-1890; fp32 13 us of 9870-10070.
constexpr int kScanned = 4096;
constexpr float kLeastRest = 0x1p-16f;       // f_i under which it stays in p
struct GradScales {                          // [N] each, but for all [1]
  float *s, *row, *at_target, *lse, *all;
};
template <typename T>
__global__ __launch_bounds__(256) void k_grad_scales(const float* __restrict__ g, const int64_t* __restrict__ target,
                                                     int64_t N, int64_t V, const T* __restrict__ h,
                                                     const T* __restrict__ W, const float* __restrict__ lse, int64_t K,
                                                     GradScales out, T* __restrict__ scaled) {
  constexpr int kEach = 16 / sizeof(T);
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t i = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (i >= N) return;
  const float gi = g[i];
  const int64_t tgt = target[i];
  const bool live = tgt >= 0 && tgt < V && gi != 0.f;
  float m = 1.f;
  if constexpr (sizeof(T) == 2) {
    float G = 1.f;
    for (int64_t t0 = 0; t0 < min(N, (int64_t)kScanned); t0 += kWave) {
      const int64_t t = min(t0 + lane, N - 1);
      const float v = fabsf(g[t]);
      const uint64_t good = __ballot(target[t] >= 0 && target[t] < V && v > 0.f && v < INFINITY);
      if (good) {
        G = __uint_as_float((__float_as_uint(__shfl(v, __builtin_ctzll(good))) & 0x007FFFFFu) | 0x3F800000u);
        break;
      }
    }
    float si = 0.f, at_target = 0.f, base = 0.f;
    if (live) {
      const T* __restrict__ hi = h + i * K;
      const T* __restrict__ wt = W + tgt * K;
      float logit = 0.f;
      for (int64_t k = lane * kEach; k < K; k += kWave * kEach) {
        const v4u a = *reinterpret_cast<const v4u*>(hi + k), b = *reinterpret_cast<const v4u*>(wt + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          logit = fmaf(bf16_lo(a[j]), bf16_lo(b[j]), logit);
          logit = fmaf(bf16_hi(a[j]), bf16_hi(b[j]), logit);
        }
      }
      logit = wave_sum(logit);
      base = lse[i];
      float f = -expm1f(logit - base);
      const bool apart = f >= kLeastRest;                                  // not a NaN either
      at_target = apart ? -1.f : -f;
      if (apart) base += logf(f);
      else f = 1.f;
      const float ratio = fabsf(gi) * f / G;
      if (ratio < INFINITY) {
        float top = fmaxf(__uint_as_float(__float_as_uint(ratio) & 0x7F800000u), 0x1p-60f);   // 2^floor(log2(ratio))
        m = ratio / top;
        if (m > 1.f && top < 0x1p127f) {
          m *= 0.5f;
          top *= 2.f;
        }
        si = copysignf(top, gi);
      } else {
        si = gi;
      }
    }
    if (lane == 0) {
      out.s[i] = si;
      out.row[i] = G * m;
      out.at_target[i] = at_target;
      out.lse[i] = base;
      if (i == 0) *out.all = G;
    }
  }
  if (!scaled) return;
  const T* __restrict__ from = h + i * K;
  T* __restrict__ to = scaled + i * K;
  for (int64_t k = lane * kEach; k < K; k += kWave * kEach) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) {
      w = *reinterpret_cast<const uint4*>(from + k);
      if constexpr (sizeof(T) == 2) {
        uint32_t* e = &w.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = pack_bf16(m * bf16_lo(e[j]), m * bf16_hi(e[j]));
      }
    }
    *reinterpret_cast<uint4*>(to + k) = w;
  }
}

namespace {

constexpr int kCUs = 256;
constexpr int64_t kPieceRows = 8192;         // vocabulary entries per piece of the gradient, less where N
                                             // tokens of it would be over 2^27 values

// Tile shapes, largest first, with the time of a tile of each per element of C relative to the first that
// the type has (2048 x 32000 x 4096, every shape in turn).  Smaller tiles read LDS and the L2 more often
// for the same products, but fill the device where there are few.
struct TileShape {
  int a, b;
  float bf16, fp32;
};
constexpr TileShape kTiles[] = {{256, 256, 1.f, 0.f}, {256, 128, 1.15f, 1.f}, {128, 128, 1.3f, 1.1f}, {128, 64, 1.7f, 1.25f}};

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }
int tiles(int64_t rows, int tile) { return (int)((rows + tile - 1) / tile); }

// Shape and splits of the contraction with the least rounds of workgroups over the device: cover_a x
// cover_b elements of C, and splits up to `most`, each worth at least 16 steps.  What follows a tile's
// steps is counted in steps: 2 for an epilogue, 28 where the tile's fp32 sums are read and written
// (`sums`: a later piece adds to them, or splits are joined afterwards; 0.5 MB for a 256 x 256 tile at a
// CU's share of HBM).
struct NtPlan {
  int shape, splits;
};
NtPlan nt_plan(int64_t cover_a, int64_t cover_b, int64_t steps, int elem, int most, bool sums) {
  const int first = elem == 2 ? 0 : 1;                     // three parts of a 256 x 256 step are over LDS
  NtPlan best{first, 1};
  double least = 0;
  for (int k = first; k < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++k)
    for (int s = 1; s <= most && (s == 1 || steps / s >= 16); ++s) {
      const int64_t wgs = (int64_t)tiles(cover_a, kTiles[k].a) * tiles(cover_b, kTiles[k].b) * s;
      const double rounds = (double)((wgs + kCUs - 1) / kCUs);
      const double tile = kTiles[k].a * kTiles[k].b * (elem == 2 ? kTiles[k].bf16 : kTiles[k].fp32);
      const double cost = rounds * tile * ((double)steps / s + (sums ? 28 : s > 1 ? 14 : 2));
      if ((k == first && s == 1) || cost < least) {
        least = cost;
        best = NtPlan{k, s};
      }
    }
  return best;
}

template <typename T, int EPI>
void launch_nt(VocabTile& t, const NtPlan& plan, int64_t cover_a, int64_t cover_b, hipStream_t s) {
  t.tiles_a = tiles(cover_a, kTiles[plan.shape].a);
  t.tiles_b = tiles(cover_b, kTiles[plan.shape].b);
  t.splits = plan.splits;
  const dim3 grid((t.tiles_a * t.tiles_b + 7) / 8 * 8, plan.splits);
  if constexpr (sizeof(T) == 2) {
    switch (plan.shape) {
      case 0: hipLaunchKernelGGL((k_nt<256, 256, 2, 4, EPI>), grid, dim3(512), 0, s, t); break;
      case 1: hipLaunchKernelGGL((k_nt<256, 128, 4, 2, EPI>), grid, dim3(512), 0, s, t); break;
      case 2: hipLaunchKernelGGL((k_nt<128, 128, 2, 2, EPI>), grid, dim3(256), 0, s, t); break;
      default:
        if ((EPI == kLoss || EPI == kGrad) && t.tiles_a * t.tiles_b <= kCUs)
          hipLaunchKernelGGL((k_nt<128, 64, 2, 2, EPI, EPI == kLoss || EPI == kGrad ? 4 : 2>), grid, dim3(256), 0, s, t);
        else
          hipLaunchKernelGGL((k_nt<128, 64, 2, 2, EPI>), grid, dim3(256), 0, s, t);
        break;
    }
  } else {
    switch (plan.shape) {
      case 1: hipLaunchKernelGGL((k_nt_split<256, 128, 4, 2, EPI>), grid, dim3(512), 0, s, t); break;
      case 2: hipLaunchKernelGGL((k_nt_split<128, 128, 2, 4, EPI>), grid, dim3(512), 0, s, t); break;
      default: hipLaunchKernelGGL((k_nt_split<128, 64, 4, 2, EPI>), grid, dim3(512), 0, s, t); break;
    }
  }
}

int64_t steps_of(int64_t k, int elem) { return (k * elem + 127) / 128; }

struct LossPlan {
  NtPlan nt;
  size_t part, tlogit, total;
};
LossPlan loss_plan(int64_t N, int64_t V, int64_t K, int elem) {
  LossPlan p;
  p.nt = nt_plan(V, N, steps_of(K, elem), elem, 1, false);
  p.part = 0;
  p.tlogit = up256((size_t)tiles(V, kTiles[p.nt.shape].a) * N * sizeof(float2));
  p.total = p.tlogit + up256((size_t)N * 4);
  return p;
}

struct GradPlan {
  int64_t piece;
  int pieces;
  NtPlan hidden;
  size_t p, acc, scales, scaled, total;
};
GradPlan grad_plan(int64_t N, int64_t V, int64_t K, int elem) {
  GradPlan g;
  const int64_t fit = std::min((int64_t(1) << 27) / N, (int64_t(1) << 30) / (K * elem)) / 256 * 256;
  const int64_t most = std::max<int64_t>(256, std::min<int64_t>(kPieceRows, fit));
  g.pieces = (int)((V + most - 1) / most);
  g.piece = ((V + g.pieces - 1) / g.pieces + 255) / 256 * 256;
  g.pieces = (int)((V + g.piece - 1) / g.piece);
  g.hidden = nt_plan(K, N, steps_of(std::min(g.piece, V), elem), elem, 8, g.pieces > 1);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
  g.p = take((size_t)N * g.piece * elem);
  g.acc = take(g.pieces > 1 || g.hidden.splits > 1 ? (size_t)g.hidden.splits * N * K * 4 : 0);
  g.scales = take(elem == 2 ? ((size_t)4 * N + 1) * 4 : 0);
  g.scaled = take((size_t)N * K * elem);
  g.total = at;
  return g;
}

template <typename T>
hipError_t loss_t(const VocabArgs& a, hipStream_t s) {
  const LossPlan p = loss_plan(a.N, a.V, a.K, sizeof(T));
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  VocabTile t{};
  t.a = a.W; t.b = a.h;
  t.rows_a = a.V; t.rows_b = a.N;
  t.k = t.lda = t.ldb = a.K;
  t.target = a.target;
  t.part = reinterpret_cast<float2*>(ws + p.part);
  t.tlogit = reinterpret_cast<float*>(ws + p.tlogit);
  t.V = a.V; t.N = a.N;
  launch_nt<T, kLoss>(t, p.nt, a.V, a.N, s);
  hipLaunchKernelGGL(k_loss_join, dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, s, t.part, t.tlogit, a.target, a.N, a.V,
                     t.tiles_a, a.loss, a.lse_out);
  return hipGetLastError();
}

template <typename T>
hipError_t grad_t(const VocabArgs& a, hipStream_t s) {
  const GradPlan q = grad_plan(a.N, a.V, a.K, sizeof(T));
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  T* p = reinterpret_cast<T*>(ws + q.p);
  float* acc = reinterpret_cast<float*>(ws + q.acc);
  const T* W = static_cast<const T*>(a.W);
  const float *factor = a.g, *lse = a.lse, *at_target = nullptr, *row_scale = nullptr, *all_scale = nullptr;
  float* sc = reinterpret_cast<float*>(ws + q.scales);
  const GradScales out{sc, sc + a.N, sc + 2 * a.N, sc + 3 * a.N, sc + 4 * a.N};
  T* h = a.dW ? reinterpret_cast<T*>(ws + q.scaled) : nullptr;
  if (sizeof(T) == 2) {
    factor = out.s;
    lse = out.lse;
    at_target = out.at_target;
    row_scale = out.row;
    all_scale = out.all;
  }
  if (sizeof(T) == 2 || h)
    hipLaunchKernelGGL((k_grad_scales<T>), dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, s, a.g, a.target, a.N, a.V,
                       static_cast<const T*>(a.h), W, a.lse, a.K, out, h);
  for (int k = 0; k < q.pieces; ++k) {
    const int64_t v0 = k * q.piece, rows = std::min(q.piece, a.V - v0), ldp = up64(rows);
    VocabTile t{};
    t.a = W + v0 * a.K; t.b = a.h;
    t.rows_a = rows; t.rows_b = a.N;
    t.k = t.lda = t.ldb = a.K;
    t.target = a.target; t.lse = lse; t.g = factor; t.at_target = at_target;
    t.p = p; t.ldp = ldp;
    t.v0 = v0; t.V = a.V; t.N = a.N;
    launch_nt<T, kGrad>(t, nt_plan(ldp, a.N, steps_of(a.K, sizeof(T)), sizeof(T), 1, false), ldp, a.N, s);
    if (a.dh) {
      VocabTile d{};
      d.a = W + v0 * a.K; d.b = p;
      d.rows_a = a.K; d.rows_b = a.N;
      d.k = rows; d.lda = a.K; d.ldb = ldp;
      d.acc = acc;
      d.row_scale = row_scale;
      d.out = a.dh;
      d.first = k == 0; d.last = k == q.pieces - 1;
      launch_nt<T, kHidden>(d, q.hidden, a.K, a.N, s);
      if (d.last && q.hidden.splits > 1)
        hipLaunchKernelGGL((k_hidden_join<T>), dim3((unsigned)((a.N * a.K / 4 + 255) / 256)), dim3(256), 0, s, acc,
                           row_scale, static_cast<T*>(a.dh), a.N * a.K, a.K, q.hidden.splits);
    }
    if (a.dW) {
      VocabTile d{};
      d.a = h; d.b = p;
      d.all_scale = all_scale;
      d.rows_a = a.K; d.rows_b = rows;
      d.k = a.N; d.lda = a.K; d.ldb = ldp;
      d.out = static_cast<T*>(a.dW) + v0 * a.K;
      launch_nt<T, kWeight>(d, nt_plan(a.K, rows, steps_of(a.N, sizeof(T)), sizeof(T), 1, false), a.K, rows, s);
    }
  }
  return hipGetLastError();
}

}  // namespace

size_t vocab_loss_workspace_bytes(int64_t N, int64_t V, int64_t K, int bf16) {
  return loss_plan(N, V, K, bf16 ? 2 : 4).total;
}
size_t vocab_loss_backward_workspace_bytes(int64_t N, int64_t V, int64_t K, int bf16) {
  return grad_plan(N, V, K, bf16 ? 2 : 4).total;
}
hipError_t launch_vocab_loss(const VocabArgs& a, hipStream_t s) { return a.bf16 ? loss_t<uint16_t>(a, s) : loss_t<float>(a, s); }
hipError_t launch_vocab_loss_backward(const VocabArgs& a, hipStream_t s) {
  return a.bf16 ? grad_t<uint16_t>(a, s) : grad_t<float>(a, s);
}

}  // namespace f2i
