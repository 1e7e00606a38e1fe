// Softmax cross entropy over a large vocabulary without keeping the logits, and its gradient.
//
//     l_iv = <h_i, W_v>,  lse_i = log sum_v exp l_iv,  loss_i = lse_i - l_{i, t_i}
//     p_iv = g_i (exp(l_iv - lse_i) - [v = t_i]),  dh_i = sum_v p_iv W_v,  dW_v = sum_i p_iv h_i
//
// One tiled product C = A B^T (rows of A and B contiguous along the contraction) on the matrix
// cores does all the work; what differs is what happens to a finished tile:
//   logits   A = W, B = h: each tile is reduced on chip to a (maximum, sum of exponentials) pair
//            per token, and the target's logit is picked out; no logit is stored.
//   p        the same product again for a piece of the vocabulary: p is rounded to the inputs' dtype
//            and stored twice, as [token][v] and as [v][token] (the two products below contract v
//            and the token).  For bf16 inputs this rounding (2^-8 of each p) adds about as much to
//            dh and dW as their own final rounding to bf16.
//   dh       A = W^T piece, B = p: fp32 sums over the pieces, rounded once at the end.
//   dW       A = h^T, B = p^T: rows of the piece, rounded once.
// Sums are fp32; a C tile has the A rows in its accumulator rows, so a lane holds four consecutive
// vocabulary entries (or hidden columns) of one token (or vocabulary row).
#include <algorithm>

#include "common.hpp"

namespace f2i {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

namespace {

enum { kLoss = 0, kGrad = 1, kHidden = 2, kWeight = 3 };

// acc += a b on the matrix cores, one 16-byte operand per lane.  The accumulator is tied to its own
// accumulation registers: left to itself the compiler moves the 256 of a 128 x 128 wave tile about,
// which cost a third of the time.  (Consecutive calls use different accumulators, and settle()
// separates the last one from whatever reads them.)
template <typename T>
__device__ __forceinline__ void mma(v4f& acc, const v4u& a, const v4u& b) {
  if constexpr (sizeof(T) == 2) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      asm volatile("v_mfma_f32_16x16x4_f32 %0, %1, %2, %0" : "+a"(acc) : "v"(a[e]), "v"(b[e]));
  }
}
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// exp(x) for x <= 0: off by |x| 2^-24 of itself, which in sum_v exp(l_v - top) comes to at most
// log(V) 2^-24 of the sum (the mean distance from the maximum under the softmax is at most log V).
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// exp(l - top), 1 where both are the same infinity.
__device__ __forceinline__ float exp_off(float l, float top) { return l == top ? 1.f : fast_exp(l - top); }

}  // namespace

// What the epilogues need.
struct VocabTile {
  int64_t rows_a, rows_b;       // rows of A and B
  int64_t k;                    // contraction (a multiple of 128 bytes of T)
  int64_t lda, ldb;
  const void* a;
  const void* b;
  const int64_t* target;        // [N]
  const float* lse;             // [N] (kGrad)
  const float* g;               // [N] (kGrad)
  float2* part;                 // [row tile of A][N] (kLoss)
  float* tlogit;                // [N] (kLoss)
  void* p;                      // [N][ldp] (kGrad)
  void* pt;                     // [ldp][ldt] (kGrad)
  float* acc;                   // [rows_b][rows_a] fp32 running sums (kHidden)
  void* out;                    // [rows_b][rows_a] (kHidden on the last piece, kWeight)
  int64_t v0, V;                // first vocabulary entry of A, vocabulary size
  int64_t N, ldp, ldt;
  int first, last;              // piece
  int tiles_a, tiles_b;
};

// Workgroup: a BM x BN tile of C, WA x WB waves, each BM/WA x BN/WB.  The contraction runs in steps of
// 128 bytes of every row (a whole cache line: 64-byte pieces halved the L2's throughput), double
// buffered in LDS, each step multiplied in two halves.  While a half is multiplied (its operands
// already in registers) the wave reads the next half's operands from LDS; once a step's second half
// is in registers everywhere (the step's one barrier), the copies of the step after next go straight
// into its buffer and have the rest of this step and half of the next one to land.  16-byte segment sg
// of row R lies in place sg ^ (R % 8) of its 128 bytes: any eight neighbouring lanes of an operand read
// cover all banks once.  Rows past the end of a matrix read as 0; past the last step the copies repeat
// it, which nothing reads.
template <typename T, int BM, int BN, int WA, int WB, int EPI>
__global__ __launch_bounds__(64 * WA * WB, 1) void k_nt(VocabTile t) {
  constexpr int kWaves = WA * WB;
  constexpr int FA = BM / WA / 16, FB = BN / WB / 16;
  constexpr int kBlocks = (BM + BN) / 8;                  // 1 KB copies (8 rows) per step
  static_assert(kBlocks % kWaves == 0 && BM % 8 == 0, "whole copies per wave");
  constexpr int kMine = kBlocks / kWaves;
  constexpr int kStep = (BM + BN) * 128;
  __shared__ __align__(16) uint8_t s_buf[2 * kStep];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int wa = wave / WB, wb = wave % WB;
  // Workgroups go to the eight XCDs in turn; each XCD takes a contiguous run of tiles with the B tiles
  // innermost, so the A rows of a run are fetched into one L2 only.
  const int per_xcd = (t.tiles_a * t.tiles_b + 7) / 8;
  const int tile = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || tile >= t.tiles_a * t.tiles_b) return;
  const int ta = tile / t.tiles_b, tb = tile % t.tiles_b;
  const int64_t a0 = (int64_t)ta * BM, b0 = (int64_t)tb * BN;
  const int64_t ra = min((int64_t)BM, t.rows_a - a0), rb = min((int64_t)BN, t.rows_b - b0);
  const __amdgpu_buffer_rsrc_t rs_a =
      range_rsrc(static_cast<const T*>(t.a) + a0 * t.lda, max(ra, (int64_t)0) * t.lda * sizeof(T));
  const __amdgpu_buffer_rsrc_t rs_b =
      range_rsrc(static_cast<const T*>(t.b) + b0 * t.ldb, max(rb, (int64_t)0) * t.ldb * sizeof(T));
  uint32_t off[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int R = (wave * kMine + i) * 8 + (lane >> 3), sg = (lane & 7) ^ (R & 7);
    off[i] = (uint32_t)(((R < BM ? R * t.lda : (R - BM) * t.ldb)) * sizeof(T)) + 16 * sg;
  }
  const int steps = (int)(t.k * sizeof(T) / 128);
  // this wave's copy i of a step
  auto copy = [&](int step, int buf, int i) {
    const int koff = min(step, steps - 1) * 128;
    const int blk = wave * kMine + i;
    const uint32_t voff = off[i];
    if (blk * 8 < BM)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_a, (lds_ptr_t)(s_buf + buf * kStep + blk * 1024), 16, voff, koff, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_b, (lds_ptr_t)(s_buf + buf * kStep + blk * 1024), 16, voff, koff, 0, 0);
  };
  int at_a[2], at_b[2];                                   // operand offsets of the two halves
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = c * 128 + ((4 * h + g) ^ (c & 7)) * 16;
    at_a[h] = wa * FA * 2048 + at;
    at_b[h] = BM * 128 + wb * FB * 2048 + at;
  }
  v4f acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  v4u fa[2][FA], fb[2][FB];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < kMine; ++i) copy(r, r, i);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((kMine & 15) | ((kMine >> 4) << 14) | 0xF70);   // step 0 has landed
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < FA; ++i) fa[0][i] = *reinterpret_cast<const v4u*>(s_buf + at_a[0] + i * 2048);
#pragma unroll
  for (int j = 0; j < FB; ++j) fb[0][j] = *reinterpret_cast<const v4u*>(s_buf + at_b[0] + j * 2048);
  for (int s = 0; s < steps; ++s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // FA groups of FB products; ahead of each group its share of the reads and copies
      const uint8_t* next = s_buf + ((s + h) & 1) * kStep;
#pragma unroll
      for (int i = 0; i < FA; ++i) {
        fa[h ^ 1][i] = *reinterpret_cast<const v4u*>(next + at_a[h ^ 1] + i * 2048);
#pragma unroll
        for (int j = i * FB / FA; j < (i + 1) * FB / FA; ++j)
          fb[h ^ 1][j] = *reinterpret_cast<const v4u*>(next + at_b[h ^ 1] + j * 2048);
        if (h == 1) {
#pragma unroll
          for (int k = i * kMine / FA; k < (i + 1) * kMine / FA; ++k) copy(s + 2, s & 1, k);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < FB; ++j) mma<T>(acc[i][j], fa[h][i], fb[h][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (h == 0) {
        // this wave holds the step's second half, and its copies of the next step have landed
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x70);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0);                           // no copy outlives its buffer
  settle();
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j) asm volatile("" : "+a"(acc[i][j]));   // read only after settle()

  const int64_t va = a0 + wa * FA * 16 + 4 * g;            // this lane's first A row
  const int64_t nb = b0 + wb * FB * 16 + c;                // its first B row
  if constexpr (EPI == kLoss) {
    // The pairs of the tile's waves take over the operand buffers.  (They are not an array of their own:
    // with two arrays in LDS the compiler no longer knows that an operand read cannot meet a copy in
    // flight and waits for every copy before every read, which doubled the time.)
    __syncthreads();                                       // every wave's copies have landed
    float2(*s_red)[BN] = reinterpret_cast<float2(*)[BN]>(s_buf);
    static_assert(WA * BN * sizeof(float2) <= sizeof(s_buf), "the pairs fit");
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
    for (int k = tid; k < BN; k += 64 * kWaves) {
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
    T* __restrict__ pt = static_cast<T*>(t.pt);
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int64_t tok = nb + 16 * j;
      if (tok >= t.ldt) continue;
      const int64_t tgt = tok < t.N ? t.target[tok] : -1;
      const bool live = tgt >= 0 && tgt < t.V;
      const float lse = live ? t.lse[tok] : 0.f, gi = live ? t.g[tok] : 0.f;
#pragma unroll
      for (int i = 0; i < FA; ++i) {
        const int64_t r = va + 16 * i;                     // row within the piece
        if (r >= t.ldp) continue;
        T o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t v = t.v0 + r + e;
          float x = 0.f;
          if (live && v < t.V && r + e < t.rows_a) x = gi * (expf(acc[i][j][e] - lse) - (v == tgt ? 1.f : 0.f));
          store_out(o, e, x);
          pt[(r + e) * t.ldt + tok] = o[e];
        }
        if (tok < t.N) {
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(p + tok * t.ldp + r) =
                make_uint2(o[0] | ((uint32_t)o[1] << 16), o[2] | ((uint32_t)o[3] << 16));
          else
            *reinterpret_cast<v4f*>(p + tok * t.ldp + r) = v4f{o[0], o[1], o[2], o[3]};
        }
      }
    }
  } else {
    T* __restrict__ out = static_cast<T*>(t.out);
#pragma unroll
    for (int j = 0; j < FB; ++j) {
      const int64_t rowb = nb + 16 * j;
      if (rowb >= t.rows_b) continue;
#pragma unroll
      for (int i = 0; i < FA; ++i) {
        const int64_t col = va + 16 * i;
        if (col >= t.rows_a) continue;                     // rows_a is a multiple of 64
        const int64_t at = rowb * t.rows_a + col;
        v4f v = acc[i][j];
        if constexpr (EPI == kHidden) {
          if (!t.first) v += *reinterpret_cast<const v4f*>(t.acc + at);
          if (!t.last) {
            *reinterpret_cast<v4f*>(t.acc + at) = v;
            continue;
          }
        }
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint2*>(out + at) =
              make_uint2(f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16),
                         f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16));
        else
          *reinterpret_cast<v4f*>(out + at) = v;
      }
    }
  }
}

// Joins the tiles' pairs in order (one wave per token) into lse, and the loss from the target's logit.
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

// out [cols][ldo] = in [rows][cols] transposed, columns rows..ldo-1 zeroed.
template <typename T>
__global__ __launch_bounds__(256) void k_transpose_pad(const T* __restrict__ in, T* __restrict__ out, int64_t rows,
                                                       int64_t cols, int64_t ldo) {
  __shared__ T s[64][65];
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * 64, r0 = (int64_t)blockIdx.y * 64;
#pragma unroll
  for (int j = 0; j < 64; j += 4) {
    const int64_t rr = r0 + ty + j;
    s[ty + j][tx] = rr < rows ? in[rr * cols + c0 + tx] : T(0);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 64; j += 4) out[(c0 + ty + j) * ldo + r0 + tx] = s[tx][ty + j];
}

namespace {

constexpr int kWA = 2, kWB = 4;
constexpr int kTileA = 256, kTileB = 256;
constexpr int64_t kPieceRows = 8192;         // vocabulary entries per piece of the gradient, less where N
                                             // tokens of it would be over 2^27 values

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }
int tiles(int64_t rows, int tile) { return (int)((rows + tile - 1) / tile); }

template <typename T, int EPI>
void launch_nt(VocabTile& t, int64_t cover_a, int64_t cover_b, hipStream_t s) {
  t.tiles_a = tiles(cover_a, kTileA);
  t.tiles_b = tiles(cover_b, kTileB);
  hipLaunchKernelGGL((k_nt<T, kTileA, kTileB, kWA, kWB, EPI>), dim3((t.tiles_a * t.tiles_b + 7) / 8 * 8), dim3(64 * kWA * kWB), 0, s, t);
}

struct LossPlan {
  size_t part, tlogit, total;
};
LossPlan loss_plan(int64_t N, int64_t V) {
  LossPlan p;
  p.part = 0;
  p.tlogit = up256((size_t)tiles(V, kTileA) * N * sizeof(float2));
  p.total = p.tlogit + up256((size_t)N * 4);
  return p;
}

struct GradPlan {
  int64_t piece, ldt;
  int pieces;
  size_t p, pt, wt, ht, acc, total;
};
GradPlan grad_plan(int64_t N, int64_t V, int64_t K, int elem) {
  GradPlan g;
  const int64_t most = std::max<int64_t>(256, std::min<int64_t>(kPieceRows, (int64_t(1) << 27) / N / 256 * 256));
  g.pieces = (int)((V + most - 1) / most);
  g.piece = (V + g.pieces - 1) / g.pieces;
  g.piece = (g.piece + 255) / 256 * 256;
  g.pieces = (int)((V + g.piece - 1) / g.piece);
  g.ldt = up64(N);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
  g.p = take((size_t)N * g.piece * elem);
  g.pt = take((size_t)g.piece * g.ldt * elem);
  g.wt = take((size_t)K * g.piece * elem);
  g.ht = take((size_t)K * g.ldt * elem);
  g.acc = take(g.pieces > 1 ? (size_t)N * K * 4 : 0);
  g.total = at;
  return g;
}

template <typename T>
hipError_t loss_t(const VocabArgs& a, hipStream_t s) {
  const LossPlan p = loss_plan(a.N, a.V);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  VocabTile t{};
  t.a = a.W; t.b = a.h;
  t.rows_a = a.V; t.rows_b = a.N;
  t.k = t.lda = t.ldb = a.K;
  t.target = a.target;
  t.part = reinterpret_cast<float2*>(ws + p.part);
  t.tlogit = reinterpret_cast<float*>(ws + p.tlogit);
  t.V = a.V; t.N = a.N;
  launch_nt<T, kLoss>(t, a.V, a.N, s);
  hipLaunchKernelGGL(k_loss_join, dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, s, t.part, t.tlogit, a.target, a.N, a.V,
                     t.tiles_a, a.loss, a.lse_out);
  return hipGetLastError();
}

template <typename T>
hipError_t grad_t(const VocabArgs& a, hipStream_t s) {
  const GradPlan q = grad_plan(a.N, a.V, a.K, sizeof(T));
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  T* p = reinterpret_cast<T*>(ws + q.p);
  T* pt = reinterpret_cast<T*>(ws + q.pt);
  T* wt = reinterpret_cast<T*>(ws + q.wt);
  T* ht = reinterpret_cast<T*>(ws + q.ht);
  const T* W = static_cast<const T*>(a.W);
  const T* h = static_cast<const T*>(a.h);
  if (a.dW)
    hipLaunchKernelGGL((k_transpose_pad<T>), dim3((unsigned)(a.K / 64), (unsigned)(q.ldt / 64)), dim3(256), 0, s, h, ht,
                       a.N, a.K, q.ldt);
  for (int k = 0; k < q.pieces; ++k) {
    const int64_t v0 = k * q.piece, rows = std::min(q.piece, a.V - v0), ldp = up64(rows);
    VocabTile t{};
    t.a = W + v0 * a.K; t.b = h;
    t.rows_a = rows; t.rows_b = a.N;
    t.k = t.lda = t.ldb = a.K;
    t.target = a.target; t.lse = a.lse; t.g = a.g;
    t.p = p; t.pt = pt; t.ldp = ldp; t.ldt = q.ldt;
    t.v0 = v0; t.V = a.V; t.N = a.N;
    launch_nt<T, kGrad>(t, ldp, q.ldt, s);
    if (a.dh) {
      hipLaunchKernelGGL((k_transpose_pad<T>), dim3((unsigned)(a.K / 64), (unsigned)(ldp / 64)), dim3(256), 0, s,
                         W + v0 * a.K, wt, rows, a.K, ldp);
      VocabTile d{};
      d.a = wt; d.b = p;
      d.rows_a = a.K; d.rows_b = a.N;
      d.k = d.lda = d.ldb = ldp;
      d.acc = reinterpret_cast<float*>(ws + q.acc);
      d.out = a.dh;
      d.first = k == 0; d.last = k == q.pieces - 1;
      launch_nt<T, kHidden>(d, a.K, a.N, s);
    }
    if (a.dW) {
      VocabTile d{};
      d.a = ht; d.b = pt;
      d.rows_a = a.K; d.rows_b = rows;
      d.k = d.lda = d.ldb = q.ldt;
      d.out = static_cast<T*>(a.dW) + v0 * a.K;
      launch_nt<T, kWeight>(d, a.K, rows, s);
    }
  }
  return hipGetLastError();
}

}  // namespace

size_t vocab_loss_workspace_bytes(int64_t N, int64_t V, int64_t K, int bf16) {
  (void)K;
  (void)bf16;
  return loss_plan(N, V).total;
}
size_t vocab_loss_backward_workspace_bytes(int64_t N, int64_t V, int64_t K, int bf16) {
  return grad_plan(N, V, K, bf16 ? 2 : 4).total;
}
hipError_t launch_vocab_loss(const VocabArgs& a, hipStream_t s) { return a.bf16 ? loss_t<uint16_t>(a, s) : loss_t<float>(a, s); }
hipError_t launch_vocab_loss_backward(const VocabArgs& a, hipStream_t s) {
  return a.bf16 ? grad_t<uint16_t>(a, s) : grad_t<float>(a, s);
}

}  // namespace f2i
