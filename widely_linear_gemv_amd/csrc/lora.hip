// Low-rank adapters of many requests beside a shared (packed) projection, and their gradient.
//
// Rows of x come in segments; segment s covers rows [seg_start[s], seg_start[s+1]) and uses adapter
// a = seg_adapter[s] (outside [0, L): none, its rows are not touched):
//     h_i = A_a x_i                      (rank r)
//     y_i = base_i + alpha_a B_a h_i
// and, with dy given, dh_i = alpha_a B_a^T dy_i, dx_i = dx_base_i + A_a^T dh_i,
//     dA_a = sum_i dh_i x_i^T,  dB_a = sum_i alpha_a dy_i h_i^T   (sums over the rows of adapter a).
//
// Two products carry everything.  "Reduce" (k_reduce) contracts the long axis: h from x and A, dh
// from dy and a transposed copy of B.  "Expand" (k_expand) contracts the rank: y from h and B, dx
// from dh and a transposed copy of A.  Both put the adapter matrix in the A operand and 16 rows of
// x (or h) in the B operand of a 16x16 matrix-core tile, so a column of the tile is one row of x:
// rows of different requests never mix, and a NaN or infinity in one request's row or adapter stays
// in that request's outputs.  A tile that holds rows of several adapters is multiplied once per
// adapter, each time storing the columns that belong to it.
//
// Precision: bf16 products are exact in fp32 and sums are fp32.  h stays fp32 between the two
// products; for bf16 adapters k_expand splits it into bf16 parts (two for a bf16 y: off by at most
// 2^-16 of each h, far under y's own rounding of 2^-8; three for an fp32 y: off by at most 2^-24)
// that take neighbouring places of the contraction, so the matrix cores still run at the bf16 rate.
// fp32 inputs use the fp32 matrix instruction throughout.
#include <algorithm>
#include <type_traits>

#include "tiles.hpp"

namespace f2i {

namespace {

// A loaded group of which only the first `have` elements count: the others as 0.  (Whole words: `have` is
// even for bf16, or at least the kGroup.)
template <typename T>
__device__ __forceinline__ v4u first_of(v4u w, int64_t have) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k * (4 / (int)sizeof(T)) >= have) w[k] = 0;
  return w;
}

// kGroup consecutive elements at p, one by one; elements at or past `have` read as 0.
template <typename T>
__device__ __forceinline__ v4u load_group(const T* __restrict__ p, int64_t have) {
  static_assert(sizeof(T) == 2, "fp32 rows hold whole words");
  uint32_t e[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = k < have ? p[k] : 0;
  return v4u{e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16)};
}

// The segments that meet rows [t0, t1), have rows and an adapter, and are this workgroup's share
// (s % Q == q), one after another.  64 segments at a time sit in the lanes' registers (one round of
// loads for up to 64 segments); with more, the first chunk is found by comparing 64 offsets at a time.
// Every lane of the wave gets the same answers.
struct Segments {
  const int32_t* start;
  const int32_t* adapter;
  int S, L, t0, t1, q, Q, lane;
  int at;             // first segment of the chunk in registers
  int st, en, ad;     // this lane's segment
  uint64_t left;      // segments of the chunk still to visit
  bool more;

  __device__ __forceinline__ void load() {
    const int s = at + lane;
    st = start[min(s, S)];
    en = start[min(s + 1, S)];
    ad = adapter[min(s, S - 1)];
    left = __ballot(s < S && en > t0 && st < t1 && en > st && s % Q == q && ad >= 0 && ad < L);
    more = at + kWave < S && __ballot(s < S && st >= t1) == 0;
  }
  __device__ __forceinline__ Segments(const int32_t* start_, const int32_t* adapter_, int S_, int L_, int t0_, int t1_,
                                      int q_, int Q_, int lane_)
      : start(start_), adapter(adapter_), S(S_), L(L_), t0(t0_), t1(t1_), q(q_), Q(Q_), lane(lane_), at(0) {
    for (int len = S; len > kWave;) {                  // the first segment whose end lies past t0 is in [at, at + len)
      const int stride = (len + kWave - 1) / kWave;
      const uint64_t past = __ballot(start[min(at + (lane + 1) * stride, S)] > t0);
      const int k = past ? __builtin_ctzll(past) : kWave - 1;
      at = min(at + k * stride, S - 1);
      len = min(stride, S - at);
    }
    load();
  }
  // The next segment: rows [lo, hi) of the tile and the adapter a.
  __device__ __forceinline__ bool next(int& lo, int& hi, int& a) {
    while (left == 0) {
      if (!more) return false;
      at += kWave;
      load();
    }
    const int b = __builtin_ctzll(left);
    left &= left - 1;
    lo = max(__builtin_amdgcn_readlane(st, b), t0);
    hi = min(__builtin_amdgcn_readlane(en, b), t1);
    a = __builtin_amdgcn_readlane(ad, b);
    return true;
  }
};

constexpr int kRows = 16;              // rows of x per tile
// Parts that the fp32 factors of the outer sums are split into (their results are fp32).
template <typename T>
constexpr int kFactorParts = sizeof(T) == 4 ? 1 : 3;
// Parts that h is split into for adapters of type T and outputs of type YT.
template <typename T, typename YT>
constexpr int expand_parts() { return sizeof(T) == 4 ? 1 : (sizeof(YT) == 2 ? 2 : 3); }
constexpr int kReduceWaves = 4;
// How an output's ranks lie in memory: whole 16-byte groups, whole words (read as groups, the words past
// the last rank set to 0), or neither (an odd rank of bf16: element by element).
enum { kGroups = 0, kWords = 1, kHalfWords = 2 };

}  // namespace

// ------------------------------------------------------------------------------ reduce ----

// Bound by latency for few rows (one row of 4096, rank 16: 3.9 us; 16 rows with an adapter each, three
// projections, 6 MB of adapters: 5.4 us), so the contraction is cut into chunks until some
// 1024 workgroups load at once and every wave has its loads in flight together.
//
// Workgroup: 16 TR rows x one chunk of the contraction x the tile's segments s with s % Q == q; its
// four waves take a quarter of the chunk each and join in LDS.  Output: fp32 partial sums
// part[chunk][row][rp], each (chunk, row) written by exactly one workgroup (the one whose segment
// holds the row); rows without an adapter are not written.  Loads are range-checked buffer loads, all of
// U steps issued before the first product, and U more while those are multiplied.  VEC: rows of x are
// whole 16-byte groups; else a group may reach into the next row (rows are even: whole words) and the
// words past the row's end, whatever they are, count as 0.
template <typename T, int RT, int TR, bool VEC>
__global__ __launch_bounds__(64 * kReduceWaves) void k_reduce(LoraReduceGroup grp, const int32_t* __restrict__ seg_start,
                                                              const int32_t* __restrict__ seg_adapter, int S, int L,
                                                              int N, int r, int Q) {
  constexpr int G = Mma<T>::kGroup, kStep = 4 * G;
  constexpr int U = TR > 1 || RT > 4 ? 1 : (RT > 2 ? 2 : 4);   // steps loaded together
  constexpr int kTile = kRows * TR;
  __shared__ __align__(16) float s_part[kReduceWaves][kTile][RT * 16 + 4];
  const LoraReduceItem& it = grp.items[blockIdx.z];
  const int chunk = blockIdx.y;
  if ((int64_t)chunk * it.chunk >= it.K) return;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = (int)(blockIdx.x / Q) * kTile, q = blockIdx.x % Q;
  const int t1 = min(t0 + kTile, N);
  const int rp = RT * 16;
  const int64_t K = it.K;
  const int per_wave = it.chunk / kReduceWaves;
  const int64_t k0 = (int64_t)chunk * it.chunk + (int64_t)wave * per_wave;
  const int64_t kend = min(k0 + per_wave, K);
  const T* __restrict__ x = static_cast<const T*>(it.x) + (int64_t)t0 * K;
  const T* __restrict__ W = static_cast<const T*>(it.W);
  // rows past N read as 0 (and reach no stored column)
  const __amdgpu_buffer_rsrc_t rs_x = range_rsrc(x, (int64_t)(t1 - t0) * K * sizeof(T));
  auto load_x = [&](int64_t k, v4u (&o)[TR]) {
    const int64_t kk = k + g * G;
#pragma unroll
    for (int t = 0; t < TR; ++t) {
      const int64_t row = 16 * t + c;
      const uint32_t voff = kk < kend ? (uint32_t)((row * K + kk) * sizeof(T)) : kNoLoad;
      o[t] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rs_x, voff, 0, 0));
      if constexpr (!VEC) o[t] = first_of<T>(o[t], kend - kk);
    }
  };

  Segments segs(seg_start, seg_adapter, S, L, t0, t1, q, Q, lane);
  int lo, hi, a;
  while (segs.next(lo, hi, a)) {
    // one adapter: r rows of ldw; ranks past r read as 0
    const __amdgpu_buffer_rsrc_t rs_w = range_rsrc(W + (int64_t)a * r * it.ldw, (int64_t)r * it.ldw * sizeof(T));
    auto load_w = [&](int64_t k, v4u (&o)[RT]) {
      const int64_t kk = k + g * G;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const uint32_t voff = kk < kend ? (uint32_t)(((t * 16 + c) * it.ldw + kk) * sizeof(T)) : kNoLoad;
        o[t] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rs_w, voff, 0, 0));
      }
    };
    v4f acc[RT][TR];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int u = 0; u < TR; ++u) acc[t][u] = v4f{0.f, 0.f, 0.f, 0.f};
    v4u xs[2][U][TR], ws[2][U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      load_x(k0 + u * kStep, xs[0][u]);
      load_w(k0 + u * kStep, ws[0][u]);
    }
    for (int64_t k = k0; k < kend; k += 2 * U * kStep) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (k + (h + 1) * U * kStep < kend) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            load_x(k + ((h + 1) * U + u) * kStep, xs[h ^ 1][u]);
            load_w(k + ((h + 1) * U + u) * kStep, ws[h ^ 1][u]);
          }
        }
        if (h == 0 || k + U * kStep < kend) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
              for (int v = 0; v < TR; ++v) acc[t][v] = Mma<T>::run(ws[h][u][t], xs[h][u][v], acc[t][v]);
        }
      }
    }
    // C: lane holds ranks 16 t + 4 g .. + 3 of row 16 v + c
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int v = 0; v < TR; ++v) *reinterpret_cast<v4f*>(&s_part[wave][16 * v + c][t * 16 + 4 * g]) = acc[t][v];
    __syncthreads();
    for (int e = threadIdx.x; e < (hi - lo) * rp; e += 64 * kReduceWaves) {
      const int row = lo + e / rp, k = e % rp;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kReduceWaves; ++w) v += s_part[w][row - t0][k];
      it.part[((int64_t)chunk * N + row) * rp + k] = k < r ? v : 0.f;
    }
    __syncthreads();
  }
}

// k_reduce for long segments and small ranks: the same work with both operands copied straight into LDS,
// 128 contiguous bytes of a row at a time (register loads in operand layout fetch 64, and kept fewer
// bytes in flight).  Each wave has a ring of four steps of its own for its quarter of the chunk, so no
// barrier is needed until the waves join.  Bound by x from HBM and the adapters from the L2: 2048 x 4096
// bf16 at rank 32, two projections, 15.0 us (from registers 22.5); dy and x of the gradient at rank 16
// 12.6 us for 33.6 MB, 2.7 TB/s.
template <typename T, int RT>
__global__ __launch_bounds__(64 * kReduceWaves, 1) void k_reduce_ring(LoraReduceGroup grp,
                                                                      const int32_t* __restrict__ seg_start,
                                                                      const int32_t* __restrict__ seg_adapter, int S,
                                                                      int L, int N, int r) {
  constexpr int kDeep = 128 / sizeof(T), RING = 4;         // contraction per step, steps in the ring
  constexpr int kCopies = 2 + 2 * RT, kStage = kCopies * 1024;
  constexpr int rp = RT * 16;
  static_assert(kCopies * (RING - 1) < 64, "the copies in flight can be counted");
  constexpr int kFlight = kCopies * (RING - 1);
  __shared__ __align__(16) uint8_t s_ring[kReduceWaves * RING * kStage];
  static_assert(sizeof(s_ring) >= sizeof(float) * kReduceWaves * kRows * (rp + 4), "the waves' sums fit");
  using X = Side<T, kRows, false>;
  using Y = Side<T, rp, false>;
  const LoraReduceItem& it = grp.items[blockIdx.z];
  const int chunk = blockIdx.y;
  if ((int64_t)chunk * it.chunk >= it.K) return;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.x * kRows, t1 = min(t0 + kRows, N);
  const int64_t K = it.K;
  const int64_t k0 = (int64_t)chunk * it.chunk + (int64_t)wave * (it.chunk / kReduceWaves);
  const int64_t kend = min(k0 + it.chunk / kReduceWaves, K);
  const int steps = (int)max((kend - k0 + kDeep - 1) / kDeep, (int64_t)0);
  const __amdgpu_buffer_rsrc_t rs_x =
      range_rsrc(static_cast<const T*>(it.x) + (int64_t)t0 * K, (int64_t)(t1 - t0) * K * sizeof(T));
  uint32_t off_x[2], off_w[2 * RT];
#pragma unroll
  for (int i = 0; i < 2; ++i) off_x[i] = X::source(i, lane, K) + (uint32_t)(k0 * sizeof(T));
#pragma unroll
  for (int i = 0; i < 2 * RT; ++i) off_w[i] = Y::source(i, lane, it.ldw) + (uint32_t)(k0 * sizeof(T));
  // contraction of this lane's 16 bytes within a step: at or past kend it reads as 0
  const int64_t mine = k0 + (((lane & 7) ^ ((lane >> 3) & 7)) * 16) / (int)sizeof(T);
  uint8_t* ring = s_ring + wave * RING * kStage;

  Segments segs(seg_start, seg_adapter, S, L, t0, t1, 0, 1, lane);
  int lo, hi, a;
  while (segs.next(lo, hi, a)) {
    const __amdgpu_buffer_rsrc_t rs_w = range_rsrc(static_cast<const T*>(it.W) + (int64_t)a * r * it.ldw,
                                                   (int64_t)r * it.ldw * sizeof(T));
    auto copy = [&](int step) {
      uint8_t* to = ring + (step & (RING - 1)) * kStage;
      const bool in = mine + (int64_t)step * kDeep < kend;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t voff = in ? off_x[i] + step * 128 : kNoLoad;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_x, (lds_ptr_t)(to + i * 1024), 16, voff, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) {
        const uint32_t voff = in ? off_w[i] + step * 128 : kNoLoad;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs_w, (lds_ptr_t)(to + 2048 + i * 1024), 16, voff, 0, 0, 0);
      }
    };
    v4f acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < RING; ++s) copy(s);
    for (int s = 0; s < steps; ++s) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt((kFlight & 15) | ((kFlight >> 4) << 14) | 0xF70);   // step s has landed
      asm volatile("" ::: "memory");
      const uint8_t* from = ring + (s & (RING - 1)) * kStage;
      v4u xs[2], ws[2][RT];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xs[h] = X::read(from, 0, h, c, g);
#pragma unroll
        for (int t = 0; t < RT; ++t) ws[h][t] = Y::read(from + 2048, t, h, c, g);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = Mma<T>::run(ws[h][t], xs[h], acc[t]);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);                  // the step's reads are done: its place is free
      asm volatile("" ::: "memory");
      copy(s + RING);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();                                       // no copy of any wave is left in the ring
    float(*s_part)[kRows][rp + 4] = reinterpret_cast<float(*)[kRows][rp + 4]>(s_ring);
#pragma unroll
    for (int t = 0; t < RT; ++t) *reinterpret_cast<v4f*>(&s_part[wave][c][t * 16 + 4 * g]) = acc[t];
    __syncthreads();
    for (int e = threadIdx.x; e < (hi - lo) * rp; e += 64 * kReduceWaves) {
      const int row = lo + e / rp, k = e % rp;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kReduceWaves; ++w) v += s_part[w][row - t0][k];
      it.part[((int64_t)chunk * N + row) * rp + k] = k < r ? v : 0.f;
    }
    __builtin_amdgcn_s_waitcnt(0);                         // only copies are counted from here on
    __syncthreads();
  }
}

// One lane's operand group for k_expand from G sums: part `part` of the bf16 split (the leading 8 bits,
// then what is left, then what is left of that), or the fp32 values.
template <typename T>
__device__ __forceinline__ v4u operand_group(const float (&h)[Mma<T>::kGroup], int part) {
  v4u o;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = __float_as_uint(h[j]);
  } else {
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // The first part is cut off, not rounded: a value past the largest bf16 would round to infinity.
      // One that is not finite is carried by the first part alone (not inf - inf).
      const bool finite = isfinite(h[j]);
      const uint32_t top = finite ? __float_as_uint(h[j]) >> 16 : (uint32_t)f32_to_bf16_rne(h[j]);
      float v = finite ? h[j] - __uint_as_float(top << 16) : 0.f;
      uint32_t w = top;
      for (int p = 1; p <= part; ++p) {
        w = f32_to_bf16_rne(v);
        v -= __uint_as_float(w << 16);
      }
      b[j] = w;
    }
    o = v4u{b[0] | (b[1] << 16), b[2] | (b[3] << 16), b[4] | (b[5] << 16), b[6] | (b[7] << 16)};
  }
  return o;
}

// G neighbouring sums of one row, the chunks' partial sums joined in order; eight chunks' loads are in
// flight together (chunks past the last read as 0).
template <int G>
__device__ __forceinline__ void join_chunks(const float* __restrict__ part, int64_t at, int64_t pitch, int nchunk,
                                            float (&v)[G]) {
  const __amdgpu_buffer_rsrc_t rs = range_rsrc(part, pitch * nchunk * 4);
#pragma unroll
  for (int j = 0; j < G; ++j) v[j] = 0.f;
  for (int c0 = 0; c0 < nchunk; c0 += 8) {
    v4f w[8][G / 4];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int j = 0; j < G / 4; ++j)
        w[c][j] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(
            rs, c0 + c < nchunk ? (uint32_t)(((c0 + c) * pitch + at + 4 * j) * 4) : kNoLoad, 0, 0));
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int j = 0; j < G; ++j) v[j] += w[c][j >> 2][j & 3];
  }
}

// The chunks' partial sums joined and scaled by the row's alpha, as operands of the products that
// read them; rows without an adapter give 0.  blockIdx.z picks the form, one wave per 64 operands:
//   0  item.groups, k_expand's: [16-row tile][step][lane], ranks along the contraction
//   1  item.factors, k_outer's: [block of 4 G rows][rank tile][part][lane], rows along the contraction
// A launch of its own pays where every workgroup of a row tile in k_expand would join the same sums: 4.8 us
// for 2048 rows of two projections at rank 32.
template <typename T>
__global__ __launch_bounds__(256) void k_reduce_join(LoraReduceGroup grp, const int32_t* __restrict__ seg_start,
                                                     const int32_t* __restrict__ seg_adapter, int S, int L, int N,
                                                     int r, int rp, int parts, int row_blocks) {
  constexpr int G = Mma<T>::kGroup;
  const LoraReduceItem& it = grp.items[blockIdx.y];
  const int lane = threadIdx.x & (kWave - 1), c = lane & 15, g = lane >> 4;
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int nchunk = (int)((it.K + it.chunk - 1) / it.chunk);
  const int64_t pitch = (int64_t)N * rp;
  if (blockIdx.z == 0) {
    const int gpp = rp / G, steps = (parts * gpp + 3) / 4;
    const int tile = unit / steps, st = unit % steps;
    const int t0 = tile * kRows;
    if (!it.groups || t0 >= N) return;
    const int grpi = st * 4 + g, part = grpi / gpp, k = (grpi % gpp) * G, row = t0 + c;
    Segments segs(seg_start, seg_adapter, S, L, t0, min(t0 + kRows, N), 0, 1, lane);
    int own = -1;
    for (int lo, hi, a; segs.next(lo, hi, a);)
      if (row >= lo && row < hi) own = a;
    float v[G];
#pragma unroll
    for (int j = 0; j < G; ++j) v[j] = 0.f;
    if (own >= 0 && part < parts) {
      const float al = it.alpha[own];
      join_chunks<G>(it.part, (int64_t)row * rp + k, pitch, nchunk, v);
#pragma unroll
      for (int j = 0; j < G; ++j) v[j] *= al;
    }
    static_cast<v4u*>(it.groups)[((int64_t)tile * steps + st) * 64 + lane] =
        part < parts ? operand_group<T>(v, part) : v4u{0, 0, 0, 0};
  } else {
    const int rts = rp / 16, rb = unit / rts, rt = unit % rts;
    if (!it.factors || rb >= row_blocks) return;
    const int row0 = rb * 4 * G, rank = rt * 16 + c;
    int own[G];
#pragma unroll
    for (int e = 0; e < G; ++e) own[e] = -1;
    if (row0 < N) {
      Segments segs(seg_start, seg_adapter, S, L, row0, min(row0 + 4 * G, N), 0, 1, lane);
      for (int lo, hi, a; segs.next(lo, hi, a);) {
#pragma unroll
        for (int e = 0; e < G; ++e)
          if (row0 + g * G + e >= lo && row0 + g * G + e < hi) own[e] = a;
      }
    }
    const __amdgpu_buffer_rsrc_t rs = range_rsrc(it.part, pitch * nchunk * 4);
    float v[G], al[G];
#pragma unroll
    for (int e = 0; e < G; ++e) {
      v[e] = 0.f;
      al[e] = own[e] >= 0 ? it.alpha[own[e]] : 0.f;
    }
    for (int ch = 0; ch < nchunk; ch += 2) {
      float w[2][G];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < G; ++e) {
          const bool ok = own[e] >= 0 && rank < r && ch + u < nchunk;
          w[u][e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
              rs, ok ? (uint32_t)(((ch + u) * pitch + (int64_t)(row0 + g * G + e) * rp + rank) * 4) : kNoLoad, 0, 0));
        }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < G; ++e) v[e] += w[u][e];
    }
#pragma unroll
    for (int e = 0; e < G; ++e) v[e] = own[e] >= 0 ? v[e] * al[e] : 0.f;
#pragma unroll
    for (int p = 0; p < kFactorParts<T>; ++p)
      static_cast<v4u*>(it.factors)[((int64_t)unit * kFactorParts<T> + p) * 64 + lane] = operand_group<T>(v, p);
  }
}

// ------------------------------------------------------------------------------ expand ----

// Workgroup: 16 TF rows x 256 outputs (64 per wave) x the segments s with s % Q == q; for each segment
// it multiplies and stores base + delta.  The rows' operand groups come from k_reduce_join (READY: long
// segments, where every workgroup of a row tile would join the same sums again) or are made here from
// the partial sums (few rows: one launch less).  base is loaded first of all, so that it arrives while
// the segments, the groups and the adapter do.
//
// The outputs of a wave's 64 are dealt to the rows i of its four output fragments f so that a lane's
// accumulators make whole 16-byte pieces of one row of y: output 16 f + i for fp32, 32 (f / 2) +
// 8 (i / 4) + 4 (f % 2) + i % 4 for bf16 (one instruction then covers 64 contiguous bytes of each row).  With long segments workgroups are ordered with the outputs innermost, so those that
// run together read and write whole rows (beside gate/up, 2048 rows: 46 us, rows innermost 55).
//
// Bound by HBM: base is read and y written once.  Beside gate/up, 2048 x 11008 bf16 twice: 46 us for 137 MB
// fetched and 89 written, 4.9 TB/s, where a copy of 1 GiB reaches 5.2; 102 MB of the fetch are needed, the
// rest is adapters that several L2s fetch.  (Stores and loads past the caches: 48.5 and 55 us.)  One
// row and one adapter, 4096 outputs, is latency: 7 us, three dependent loads deep.
template <typename T, typename YT, int TF, bool READY, int RANKS>
__global__ __launch_bounds__(256) void k_expand(LoraExpandGroup grp, const int32_t* __restrict__ seg_start,
                                                const int32_t* __restrict__ seg_adapter, int S, int L, int N, int r,
                                                int rp, int Q) {
  constexpr int G = Mma<T>::kGroup;
  constexpr int kParts = expand_parts<T, YT>();
  constexpr int kTile = kRows * TF;
  constexpr int kBase = sizeof(YT);                        // 16-byte pieces of 16 outputs
  extern __shared__ __align__(16) v4u s_frag[];            // [TF][steps][64] (not READY)
  const LoraExpandItem& it = grp.items[blockIdx.z];
  const int64_t M = it.M;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  uint32_t row_block = blockIdx.x, out_block = blockIdx.y;
  if constexpr (READY) {                                   // dispatch order: outputs innermost
    const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
    row_block = block / gridDim.y;
    out_block = block - row_block * gridDim.y;
  }
  const int64_t o_block = (int64_t)out_block * 256, o0 = o_block + wave * 64;
  if (o_block >= M) return;
  const int t0 = (int)(row_block / Q) * kTile, q = row_block % Q;
  const int t1 = min(t0 + kTile, N);
  const int gpp = rp / G;                                  // operand groups per part
  const int steps = (kParts * gpp + 3) / 4;
  const YT* base = static_cast<const YT*>(it.base);
  YT* y = static_cast<YT*>(it.y);
  // A lane's 16-byte pieces of a row of y (rows are even, so pieces are at least 4-byte aligned, which is
  // what the vector memory instructions need); 64 outputs that M cuts short go one by one.
  typedef v4u __attribute__((aligned(4))) piece_t;
  const bool yvec = o0 + 64 <= M;
  auto output = [](int f, int i) { return sizeof(YT) == 4 ? 16 * f + i : 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3); };
  auto piece = [&](int i) { return sizeof(YT) == 4 ? 16 * i + 4 * g : 32 * i + 8 * g; };   // first output of a piece
  v4u old[TF][kBase];
#pragma unroll
  for (int t = 0; t < TF; ++t)
    if (yvec) {
      const int64_t row = min(t0 + 16 * t + c, t1 - 1);
#pragma unroll
      for (int i = 0; i < kBase; ++i)
        old[t][i] = *reinterpret_cast<const piece_t*>(base + row * M + o0 + piece(i));
    }

  Segments segs(seg_start, seg_adapter, S, L, t0, t1, q, Q, lane);
  const v4u* __restrict__ groups = nullptr;                // [TF][steps][64]
  if constexpr (READY) {
    groups = static_cast<const v4u*>(it.groups) + (int64_t)(t0 / kRows) * steps * 64;
  } else {
    for (int e = threadIdx.x; e < steps * TF * 64; e += 256) {
      const int st = (e / 64) % steps, f = e / (64 * steps), l = e % 64;
      const int grpi = st * 4 + (l >> 4), part = grpi / gpp, k = (grpi % gpp) * G, row = t0 + f * 16 + (l & 15);
      // the row's adapter (every lane of the wave is here: the segments are read across lanes)
      int own = -1;
      Segments mine = segs;
      for (int lo, hi, a; mine.next(lo, hi, a);)
        if (row >= lo && row < hi) own = a;
      float v[G];
#pragma unroll
      for (int j = 0; j < G; ++j) v[j] = 0.f;
      if (part < kParts && own >= 0) {
        const float al = it.alpha[own];
        join_chunks<G>(it.part, (int64_t)row * rp + k, (int64_t)N * rp, it.nchunk, v);
#pragma unroll
        for (int j = 0; j < G; ++j) v[j] *= al;
      }
      s_frag[e] = part < kParts ? operand_group<T>(v, part) : v4u{0, 0, 0, 0};
    }
    __syncthreads();
    groups = s_frag;
  }
  if (o0 >= M) return;
  const int tiles_here = (t1 - t0 + kRows - 1) / kRows;

  int lo, hi, a;
  while (segs.next(lo, hi, a)) {
    // one adapter's outputs o0 .. : outputs past M read as 0 and are not stored
    const T* __restrict__ Wa = static_cast<const T*>(it.W) + (int64_t)a * M * r + o0 * r;
    const __amdgpu_buffer_rsrc_t rs_w = range_rsrc(Wa, (M - o0) * r * (int64_t)sizeof(T));
    v4f acc[4][TF];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int t = 0; t < TF; ++t) acc[f][t] = v4f{0.f, 0.f, 0.f, 0.f};
    // Whole steps of ranks (rp >= 4 G) are multiplied with each part of h in turn, the adapter loaded
    // once; a rank of under 4 G shares one step between the parts.
    const int passes = gpp % 4 == 0 ? kParts : 1, wsteps = gpp % 4 == 0 ? gpp / 4 : steps;
    for (int ws = 0; ws < wsteps; ++ws) {
      const int grpi = ws * 4 + g, k = (grpi % gpp) * G;
      const int have = grpi < kParts * gpp ? r - k : 0;
      v4u wa[4], hb[TF];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int o = output(f, c);
        if constexpr (RANKS != kHalfWords) {
          wa[f] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
              rs_w, have > 0 ? (uint32_t)((o * r + k) * sizeof(T)) : kNoLoad, 0, 0));
          if constexpr (RANKS == kWords) wa[f] = first_of<T>(wa[f], have);
        } else {
          wa[f] = load_group<T>(Wa + min((int64_t)o, M - 1 - o0) * r + k, have);
        }
      }
      for (int p = 0; p < passes; ++p) {
#pragma unroll
        for (int t = 0; t < TF; ++t) hb[t] = groups[(min(t, tiles_here - 1) * steps + p * wsteps + ws) * 64 + lane];
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int t = 0; t < TF; ++t) acc[f][t] = Mma<T>::run(wa[f], hb[t], acc[f][t]);
      }
    }
#pragma unroll
    for (int t = 0; t < TF; ++t) {
      const int row = t0 + 16 * t + c;
      if (row < lo || row >= hi) continue;
      const int64_t off = (int64_t)row * M + o0;
      if (yvec) {
        if constexpr (sizeof(YT) == 4) {
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const v4f b = __builtin_bit_cast(v4f, old[t][f]);
            *reinterpret_cast<piece_t*>(y + off + piece(f)) = __builtin_bit_cast(
                v4u, v4f{b[0] + acc[f][t][0], b[1] + acc[f][t][1], b[2] + acc[f][t][2], b[3] + acc[f][t][3]});
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v4u o;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const v4f& d = acc[2 * h + (w >> 1)][t];
              const int e = 2 * (w & 1);
              o[w] = pack_bf16(bf16_lo(old[t][h][w]) + d[e], bf16_hi(old[t][h][w]) + d[e + 1]);
            }
            *reinterpret_cast<piece_t*>(y + off + piece(h)) = o;
          }
        }
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (o0 + output(f, 4 * g + e) < M) {
              const int64_t i = off + output(f, 4 * g + e);
              float b;
              if constexpr (sizeof(YT) == 4) b = base[i]; else b = bf16_lo(base[i]);
              store_out(y, i, b + acc[f][t][e]);
            }
      }
    }
  }
}

// --------------------------------------------------------------------- adapter transposes ----

// Copies of the adapter matrices with their axes exchanged, for the gradient's two products:
// in [L][R][C] -> out [L][C][ldo], columns R..ldo-1 zeroed.  blockIdx.y picks the matrix.  Launch-bound
// (3.6 us for one adapter of 4096 x 16); the adapters are a fraction of the rows that meet them.
template <typename T>
__global__ __launch_bounds__(256) void k_transpose(LoraTranspose ta, LoraTranspose tb) {
  __shared__ T s[32][33];
  const LoraTranspose& m = blockIdx.y ? tb : ta;
  const int across = (int)((m.C + 31) / 32);
  const int64_t down = (m.ldo + 31) / 32;
  if (blockIdx.x >= across * down) return;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c0 = (int64_t)(blockIdx.x % across) * 32, r0 = (int64_t)(blockIdx.x / across) * 32;
  const T* __restrict__ in = static_cast<const T*>(m.in) + (int64_t)blockIdx.z * m.R * m.C;
  T* __restrict__ out = static_cast<T*>(m.out) + (int64_t)blockIdx.z * m.C * m.ldo;
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    const int64_t rr = r0 + ty + j, cc = c0 + tx;
    s[ty + j][tx] = rr < m.R && cc < m.C ? in[rr * m.C + cc] : T(0);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    const int64_t cc = c0 + ty + j, rr = r0 + tx;
    if (cc < m.C && rr < m.ldo) out[cc * m.ldo + rr] = s[tx][ty + j];
  }
}

// --------------------------------------------------------------------------- outer sums ----

// dA (dB): for adapter a, the sum over the adapter's rows of factor[row][rank] * x[row][col].
// Workgroup: 256 columns (64 per wave) x RT tiles of 16 ranks (up to four: two workgroups share the
// columns of ranks over 64) x the rows [split * span, (split + 1) * span).  Steps
// of 64 bf16 (32 fp32) rows are copied into LDS as they lie, double buffered, and transposed on the
// way into registers (A operand: columns; B operand: the factors, made by k_reduce_join with rows along
// the contraction).  Rows of other segments are neither copied (zeros stand for them) nor counted (their
// factors are masked), so a NaN in another request's row cannot reach the sum.  Splits are joined in
// order by k_outer_join (splits > 1), so the result never depends on scheduling.  2048 x 4096 bf16 twice at
// rank 16: 12 us for 33.6 MB (2.8 TB/s; register operands, read two bytes at a time, took 20.2), and 4 us
// for the join of 8 splits.
template <typename T, int RT>
__global__ __launch_bounds__(256) void k_outer(LoraOuterGroup grp, const int32_t* __restrict__ seg_start,
                                               const int32_t* __restrict__ seg_adapter, int S, int L, int N, int r,
                                               int rts, int splits, int span) {
  constexpr int G = Mma<T>::kGroup, kDeep = 8 * G;         // rows per step
  constexpr int kParts = kFactorParts<T>;
  using X = Side<T, 256, true>;
  __shared__ __align__(16) uint8_t s_x[2 * 256 * 128];
  const LoraOuterItem& it = grp.items[blockIdx.z & 1];
  const int a = (int)(blockIdx.z >> 1);
  const int64_t C = it.C;
  const int64_t c0 = (int64_t)blockIdx.x * 256;
  if (c0 >= C) return;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int split = blockIdx.y % splits, rt0 = blockIdx.y / splits * RT;
  const int t0 = split * span, t1 = min(t0 + span, N);
  uint32_t off[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) off[i] = X::source(i * 4 + wave, lane, C) + (uint32_t)(c0 * sizeof(T));
  v4f acc[4][RT];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[f][t] = v4f{0.f, 0.f, 0.f, 0.f};

  Segments segs(seg_start, seg_adapter, S, L, t0, t1, 0, 1, lane);
  int lo, hi, who;
  while (segs.next(lo, hi, who)) {
    if (who != a) continue;
    const int first = lo / kDeep * kDeep;                  // steps start at multiples of kDeep
    auto copy = [&](int row0, int buf) {
      const __amdgpu_buffer_rsrc_t rs = range_rsrc(static_cast<const T*>(it.x) + (int64_t)row0 * C,
                                                   (int64_t)max(min(kDeep, hi - row0), 0) * C * (int64_t)sizeof(T));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = row0 + ((i * 4 + wave) * 1024 + lane * 16) / (256 * (int)sizeof(T));
        const uint32_t voff = row >= lo && row < hi ? off[i] : kNoLoad;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(s_x + buf * 32768 + (i * 4 + wave) * 1024), 16, voff, 0, 0, 0);
      }
    };
    copy(first, 0);
    for (int row0 = first, buf = 0; row0 < hi; row0 += kDeep, buf ^= 1) {
      v4u fb[2][RT * kParts];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < RT * kParts; ++t)
          fb[h][t] = static_cast<const v4u*>(it.factors)[(((int64_t)(row0 / (4 * G) + h) * rts + rt0) * kParts + t) * 64 + lane];
      __builtin_amdgcn_s_waitcnt(0);                       // this wave's copies (and factors) have landed
      __syncthreads();                                     // everyone's have, and the other buffer is free
      if (row0 + kDeep < hi) copy(row0 + kDeep, buf ^ 1);
      if (row0 < lo || row0 + kDeep > hi) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = row0 + 4 * G * h + G * g;        // this lane's G rows
          uint32_t keep[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if constexpr (sizeof(T) == 4) {
              keep[w] = row + w >= lo && row + w < hi ? 0xFFFFFFFFu : 0u;
            } else {
              keep[w] = (row + 2 * w >= lo && row + 2 * w < hi ? 0xFFFFu : 0u) |
                        (row + 2 * w + 1 >= lo && row + 2 * w + 1 < hi ? 0xFFFF0000u : 0u);
            }
          }
#pragma unroll
          for (int t = 0; t < RT * kParts; ++t)
#pragma unroll
            for (int w = 0; w < 4; ++w) fb[h][t][w] &= keep[w];
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4u fa[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) fa[f] = X::read(s_x + buf * 32768, wave * 4 + f, h, c, g);
#pragma unroll
        for (int t = 0; t < RT * kParts; ++t)
#pragma unroll
          for (int f = 0; f < 4; ++f) acc[f][t / kParts] = Mma<T>::run(fa[f], fb[h][t], acc[f][t / kParts]);
      }
    }
    __syncthreads();                                       // before the next segment's first copy
  }

  // C: lane holds columns 4 g .. + 3 of fragment f at rank 16 (rt0 + t) + c
  float* __restrict__ out = it.out + ((int64_t)split * L + a) * r * C;
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int64_t col = c0 + wave * 64 + 16 * f + 4 * g;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int rank = 16 * (rt0 + t) + c;
      if (rank >= r) continue;
      if (it.rank_major) {
        if (col < C) *reinterpret_cast<v4f*>(out + (int64_t)rank * C + col) = acc[f][t];   // C = 2m: whole pieces
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < C) out[(col + e) * r + rank] = acc[f][t][e];
      }
    }
  }
}

__global__ __launch_bounds__(256) void k_outer_join(LoraOuterGroup grp, float* __restrict__ dA, float* __restrict__ dB,
                                                    int64_t rows, int splits) {
  const LoraOuterItem& it = grp.items[blockIdx.y];
  const int64_t n = rows * it.C, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2;    // C is even
  if (i >= n) return;
  const float* __restrict__ part = it.out;
  float2 v = *reinterpret_cast<const float2*>(part + i);
  for (int s = 1; s < splits; ++s) {
    const float2 w = *reinterpret_cast<const float2*>(part + (int64_t)s * n + i);
    v.x += w.x;
    v.y += w.y;
  }
  *reinterpret_cast<float2*>((blockIdx.y ? dB : dA) + i) = v;
}

// ------------------------------------------------------------------------------- launch ----

namespace {

int rank_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

// Segments of one 16-row tile are shared out over Q workgroups, Q the mean number of segments per
// tile rounded up to a power of two: with one row per request (decode) each workgroup has one
// adapter to read instead of sixteen in a row; with long segments Q is 1.
int segment_shares(int N, int S) {
  const int rows = std::min(N, kRows);
  const int64_t mean = ((int64_t)S * rows + N - 1) / N;
  int q = 1;
  while (q < mean && q < kRows) q *= 2;
  return q;
}

// Row tiles per workgroup of k_reduce: an adapter of rank over 32 is several times the bytes of 16 rows
// of x, so long segments take 64 rows to one read of it.  (For smaller ranks 64 rows measured no faster:
// rank 32, 2048 x 4096, two projections 22.5 us with 16 rows, 24.3 with 64.)
int reduce_rows(int N, int S, int r) { return segment_shares(N, S) == 1 && N >= 256 && r > 32 ? 4 : 1; }

// Whether k_reduce_ring runs: long segments and small ranks (above, operands from registers with 64 rows
// to a workgroup), whole 16-byte pieces in every row.
bool reduce_ring(int N, int S, int r, bool vec) { return vec && segment_shares(N, S) == 1 && N >= 256 && r <= 32; }

// Contraction chunk: small enough that the launch has about 1024 workgroups (k_reduce) or one per CU
// (k_reduce_ring, whose rings keep the bytes in flight: 2048 x 4096 for two projections at rank 32
// 15.0 us, with 512 workgroups 17.0, with 1024 20.1), at least 256 elements, a multiple of 256.
int reduce_chunk(int64_t K, int N, int S, int r, bool vec, int items) {
  const int tile = kRows * reduce_rows(N, S, r);
  const int64_t wgs = (int64_t)((N + tile - 1) / tile) * segment_shares(N, S) * items;
  const int64_t want = std::max<int64_t>(1, (reduce_ring(N, S, r, vec) ? 256 : 1024) / wgs);
  const int64_t chunk = (K + want - 1) / want;
  return (int)std::max<int64_t>(256, (chunk + 255) / 256 * 256);
}

int chunks(int64_t K, int chunk) { return (int)((K + chunk - 1) / chunk); }

template <typename T, int RT, int TR>
void reduce_vec(const LoraReduceGroup& grp, bool vec, dim3 grid, const int32_t* ss, const int32_t* sa, int S, int L, int N,
                int r, int Q, hipStream_t st) {
  const dim3 block(64 * kReduceWaves);
  if (vec) hipLaunchKernelGGL((k_reduce<T, RT, TR, true>), grid, block, 0, st, grp, ss, sa, S, L, N, r, Q);
  else hipLaunchKernelGGL((k_reduce<T, RT, TR, false>), grid, block, 0, st, grp, ss, sa, S, L, N, r, Q);
}

template <typename T>
void launch_reduce(const LoraReduceGroup& grp, int count, bool vec, const int32_t* ss, const int32_t* sa, int S, int L,
                   int N, int r, hipStream_t st) {
  const int Q = segment_shares(N, S), tr = reduce_rows(N, S, r), tile = kRows * tr;
  int most = 1;
  for (int k = 0; k < count; ++k) most = std::max(most, chunks(grp.items[k].K, grp.items[k].chunk));
  if (reduce_ring(N, S, r, vec)) {
    const dim3 grid((N + kRows - 1) / kRows, most, count), block(64 * kReduceWaves);
    if (r <= 16) hipLaunchKernelGGL((k_reduce_ring<T, 1>), grid, block, 0, st, grp, ss, sa, S, L, N, r);
    else hipLaunchKernelGGL((k_reduce_ring<T, 2>), grid, block, 0, st, grp, ss, sa, S, L, N, r);
    return;
  }
  const dim3 grid((N + tile - 1) / tile * Q, most, count);
  switch (rank_tiles(r) * 8 + tr) {
    case 9: reduce_vec<T, 1, 1>(grp, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    case 17: reduce_vec<T, 2, 1>(grp, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    case 33: reduce_vec<T, 4, 1>(grp, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    case 36: reduce_vec<T, 4, 4>(grp, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    case 65: reduce_vec<T, 8, 1>(grp, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    default: reduce_vec<T, 8, 4>(grp, vec, grid, ss, sa, S, L, N, r, Q, st); break;
  }
}

// Whether the rows' operand groups are made by a launch of their own (k_reduce_join).
bool ready_groups(int N, int S) { return segment_shares(N, S) == 1 && N > 64; }
int group_steps(int r, int elem, int y_bf16) {
  const int parts = elem == 4 ? 1 : (y_bf16 ? 2 : 3);
  return (parts * (16 * rank_tiles(r) / (16 / elem)) + 3) / 4;
}
size_t group_bytes(int64_t N, int r, int elem, int y_bf16) {
  return (size_t)((N + kRows - 1) / kRows) * group_steps(r, elem, y_bf16) * 1024;
}

template <typename T, typename YT, int TF, bool READY>
void expand_tf(const LoraExpandGroup& grp, int count, const int32_t* ss, const int32_t* sa, int S, int L, int N, int r,
               int Q, hipStream_t st) {
  const int rp = 16 * rank_tiles(r);
  const size_t lds = READY ? 0 : (size_t)group_steps(r, sizeof(T), sizeof(YT) == 2) * TF * 1024;
  int64_t most = 0;
  for (int k = 0; k < count; ++k) most = std::max(most, grp.items[k].M);
  const int tile = kRows * TF;
  const dim3 grid((N + tile - 1) / tile * Q, (unsigned)((most + 255) / 256), count);
  auto run = [&](auto ranks) {
    hipLaunchKernelGGL((k_expand<T, YT, TF, READY, decltype(ranks)::value>), grid, dim3(256), lds, st, grp, ss, sa, S, L, N, r,
                       rp, Q);
  };
  if (r % Mma<T>::kGroup == 0) run(std::integral_constant<int, kGroups>());
  else if (sizeof(T) == 4 || r % 2 == 0) run(std::integral_constant<int, kWords>());
  else if constexpr (sizeof(T) == 2) run(std::integral_constant<int, kHalfWords>());
}

// Rows per workgroup of k_expand: 32 where that still leaves 2048 workgroups (an adapter fragment then
// serves two row tiles), 16 otherwise.  Beside gate/up, 2048 rows: 47 us with 32, 51 with 16, 49 with
// 64; 389 fp32 rows of 1408: 5.6 us with 16, 7.6 with 32.
template <typename T, typename YT>
void launch_expand(const LoraExpandGroup& grp, int count, const int32_t* ss, const int32_t* sa, int S, int L, int N,
                   int r, hipStream_t st) {
  int64_t wgs = 0;
  for (int k = 0; k < count; ++k) wgs += (int64_t)((N + 31) / 32) * ((grp.items[k].M + 255) / 256);
  if (ready_groups(N, S) && wgs >= 2048) expand_tf<T, YT, 2, true>(grp, count, ss, sa, S, L, N, r, 1, st);
  else if (ready_groups(N, S)) expand_tf<T, YT, 1, true>(grp, count, ss, sa, S, L, N, r, 1, st);
  else expand_tf<T, YT, 1, false>(grp, count, ss, sa, S, L, N, r, segment_shares(N, S), st);
}

template <typename T>
void launch_expand_y(const LoraExpandGroup& grp, int count, int y_bf16, const int32_t* ss, const int32_t* sa, int S,
                     int L, int N, int r, hipStream_t st) {
  if (y_bf16) launch_expand<T, uint16_t>(grp, count, ss, sa, S, L, N, r, st);
  else launch_expand<T, float>(grp, count, ss, sa, S, L, N, r, st);
}

template <typename T>
void launch_join(const LoraReduceGroup& grp, int count, int y_bf16, bool factors, const int32_t* ss, const int32_t* sa,
                 int S, int L, int N, int r, hipStream_t st) {
  const int units = (N + kRows - 1) / kRows * group_steps(r, sizeof(T), y_bf16);
  const int row_blocks = factors ? (N + 8 * Mma<T>::kGroup - 1) / (8 * Mma<T>::kGroup) * 2 : 0;
  hipLaunchKernelGGL((k_reduce_join<T>), dim3((std::max(units, row_blocks * rank_tiles(r)) + 3) / 4, count, factors ? 2 : 1),
                     dim3(256), 0, st, grp, ss, sa, S, L, N, r, 16 * rank_tiles(r), sizeof(T) == 4 ? 1 : (y_bf16 ? 2 : 3),
                     row_blocks);
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

size_t lora_part_floats(int64_t K, int chunk, int64_t N, int r) { return (size_t)chunks(K, chunk) * N * 16 * rank_tiles(r); }

template <typename T>
hipError_t lora_t(const LoraArgs& p, const LoraItem* items, int count, hipStream_t st) {
  const int64_t K = 2 * p.m;
  const int chunk = reduce_chunk(K, p.N, p.S, p.r, true, count);
  const size_t part = up256(lora_part_floats(K, chunk, p.N, p.r) * 4), groups = up256(group_bytes(p.N, p.r, sizeof(T), p.y_bf16));
  const bool ready = ready_groups(p.N, p.S);
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  LoraReduceGroup red;
  LoraExpandGroup exp;
  for (int k = 0; k < count; ++k) {
    float* w = reinterpret_cast<float*>(ws + part * k);
    void* made = ready ? ws + part * count + groups * k : nullptr;
    red.items[k] = LoraReduceItem{p.x, items[k].A, w, nullptr, made, items[k].alpha, K, K, chunk};
    exp.items[k] = LoraExpandItem{w, made, items[k].B, items[k].alpha, items[k].base, items[k].y, 2 * items[k].n,
                                  chunks(K, chunk)};
  }
  launch_reduce<T>(red, count, true, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  if (ready) launch_join<T>(red, count, p.y_bf16, false, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_expand_y<T>(exp, count, p.y_bf16, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  return hipGetLastError();
}

// Row ranges of k_outer: one workgroup a CU when there are few adapters and columns, at least two steps
// each.  (Two a CU: k_outer the same 12 us at 2048 x 4096 and rank 16, its join 5.0 us instead of 4.0.)
int outer_splits(int64_t N, int64_t C, int L, int elem) {
  const int64_t wgs = (C + 255) / 256 * L * 2, step = 128 / elem;
  const int64_t want = std::max<int64_t>(1, 256 / wgs);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, N / (2 * step)));
}
// Bytes of one item's factors: row blocks of 4 G rows in whole steps.
size_t factor_bytes(int64_t N, int r, int elem) {
  const int64_t step = 128 / elem;
  return (size_t)((N + step - 1) / step) * 2 * rank_tiles(r) * (elem == 4 ? 1 : 3) * 1024;
}

struct BackwardPlan {
  int rp, chunk_x, chunk_y, splits, span;
  int64_t K, M, Mp;
  size_t part_x, part_y, fac_x, fac_y, groups, bt, at, outer_a, outer_b, total;
};

BackwardPlan backward_plan(int64_t N, int64_t m, int64_t n, int r, int L, int S, int elem) {
  BackwardPlan b;
  b.rp = 16 * rank_tiles(r);
  b.K = 2 * m;
  b.M = 2 * n;
  b.Mp = (b.M + 63) / 64 * 64;
  const bool vec = b.M * elem % 16 == 0;
  b.chunk_x = reduce_chunk(b.K, (int)N, S, r, vec, 2);
  b.chunk_y = reduce_chunk(b.M, (int)N, S, r, vec, 2);
  const int step = 128 / elem;
  b.splits = outer_splits(N, std::max(b.K, b.M), L, elem);
  b.span = (int)(((N + b.splits - 1) / b.splits + step - 1) / step * step);
  b.splits = (int)((N + b.span - 1) / b.span);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
  b.part_x = take((size_t)chunks(b.K, b.chunk_x) * N * b.rp * 4);
  b.part_y = take((size_t)chunks(b.M, b.chunk_y) * N * b.rp * 4);
  b.fac_x = take(factor_bytes(N, r, elem));
  b.fac_y = take(factor_bytes(N, r, elem));
  b.groups = take(group_bytes(N, r, elem, 0));           // an fp32 dx has the most parts
  b.bt = take((size_t)L * r * b.Mp * elem);
  b.at = take((size_t)L * b.K * r * elem);
  b.outer_a = take(b.splits > 1 ? (size_t)b.splits * L * r * b.K * 4 : 0);
  b.outer_b = take(b.splits > 1 ? (size_t)b.splits * L * r * b.M * 4 : 0);
  b.total = at;
  return b;
}

template <typename T, int RT>
void launch_outer(const LoraOuterGroup& out, const BackwardPlan& b, const LoraBackwardArgs& p, hipStream_t st) {
  const int rts = rank_tiles(p.r);
  const dim3 grid((unsigned)((std::max(b.K, b.M) + 255) / 256), b.splits * (rts / RT), 2 * p.L);
  hipLaunchKernelGGL((k_outer<T, RT>), grid, dim3(256), 0, st, out, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, rts,
                     b.splits, b.span);
}

template <typename T>
hipError_t lora_backward_t(const LoraBackwardArgs& p, hipStream_t st) {
  const BackwardPlan b = backward_plan(p.N, p.m, p.n, p.r, p.L, p.S, sizeof(T));
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  T* Bt = reinterpret_cast<T*>(ws + b.bt);
  T* At = reinterpret_cast<T*>(ws + b.at);
  const dim3 block(256);
  const LoraTranspose tb{p.B, Bt, b.M, p.r, b.Mp}, ta{p.A, At, p.r, b.K, p.r};
  const int64_t across = (p.r + 31) / 32;
  hipLaunchKernelGGL((k_transpose<T>), dim3((unsigned)(across * std::max((b.Mp + 31) / 32, (b.K + 31) / 32)), p.dx ? 2 : 1, p.L),
                     block, 0, st, tb, ta);
  const bool vec = (b.M * sizeof(T)) % 16 == 0;
  const bool ready = ready_groups(p.N, p.S);
  float* part_y = reinterpret_cast<float*>(ws + b.part_y);
  LoraReduceGroup red;
  red.items[0] = LoraReduceItem{p.x, p.A, reinterpret_cast<float*>(ws + b.part_x), ws + b.fac_x, nullptr, p.alpha, b.K, b.K, b.chunk_x};
  red.items[1] = LoraReduceItem{p.dy, Bt, part_y, ws + b.fac_y, p.dx && ready ? ws + b.groups : nullptr, p.alpha, b.M, b.Mp, b.chunk_y};
  launch_reduce<T>(red, 2, vec, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  launch_join<T>(red, 2, p.dx_bf16, true, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  if (p.dx) {
    LoraExpandGroup exp;
    exp.items[0] = LoraExpandItem{part_y, ws + b.groups, At, p.alpha, p.dx_base, p.dx, b.K, chunks(b.M, b.chunk_y)};
    launch_expand_y<T>(exp, 1, p.dx_bf16, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  }
  LoraOuterGroup out;
  float* da = b.splits > 1 ? reinterpret_cast<float*>(ws + b.outer_a) : p.dA;
  float* db = b.splits > 1 ? reinterpret_cast<float*>(ws + b.outer_b) : p.dB;
  out.items[0] = LoraOuterItem{p.x, ws + b.fac_y, da, b.K, 1};
  out.items[1] = LoraOuterItem{p.dy, ws + b.fac_x, db, b.M, 0};
  if (p.r <= 16) launch_outer<T, 1>(out, b, p, st);
  else if (p.r <= 32) launch_outer<T, 2>(out, b, p, st);
  else launch_outer<T, 4>(out, b, p, st);
  if (b.splits > 1) {
    const int64_t na = (int64_t)p.L * p.r * b.K, nb = (int64_t)p.L * p.r * b.M;
    hipLaunchKernelGGL(k_outer_join, dim3((unsigned)((std::max(na, nb) + 511) / 512), 2), block, 0, st, out, p.dA, p.dB,
                       (int64_t)p.L * p.r, b.splits);
  }
  return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int count, int64_t N, int64_t m, int r, int64_t S) {
  size_t most = 0;
  for (int items : {std::min(count, kMaxLoraItems), count % kMaxLoraItems}) {
    if (items < 1) continue;
    const int chunk = reduce_chunk(2 * m, (int)N, (int)S, r, true, items);
    // the operand groups of fp32 outputs (three parts) are the largest
    const size_t groups = std::max(group_bytes(N, r, 2, 0), group_bytes(N, r, 4, 0));
    most = std::max(most, items * (up256(lora_part_floats(2 * m, chunk, N, r) * 4) +
                                   (ready_groups((int)N, (int)S) ? up256(groups) : 0)));
  }
  return most;
}

hipError_t launch_lora(const LoraArgs& p, const LoraItem* items, int count, hipStream_t st) {
  return p.x_bf16 ? lora_t<uint16_t>(p, items, count, st) : lora_t<float>(p, items, count, st);
}

size_t lora_backward_workspace_bytes(int64_t N, int64_t m, int64_t n, int r, int L, int64_t S, int x_bf16) {
  return backward_plan(N, m, n, r, L, (int)S, x_bf16 ? 2 : 4).total;
}

hipError_t launch_lora_backward(const LoraBackwardArgs& p, hipStream_t st) {
  return p.x_bf16 ? lora_backward_t<uint16_t>(p, st) : lora_backward_t<float>(p, st);
}

}  // namespace f2i
