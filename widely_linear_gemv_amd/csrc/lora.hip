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

#include "common.hpp"

namespace f2i {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

namespace {

// One 16-byte operand per lane (row or column lane & 15, contraction group lane >> 4).
template <typename T> struct Mma;
template <> struct Mma<uint16_t> {
  static constexpr int kGroup = 8;     // contraction elements per lane and step
  __device__ static v4f run(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};
template <> struct Mma<float> {
  static constexpr int kGroup = 4;
  __device__ static v4f run(v4u a, v4u b, v4f c) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
};

// kGroup consecutive elements at p; elements at or past `have` read as 0.  VEC: p is 16-byte
// aligned and `have` is a multiple of kGroup (or <= 0).
template <typename T, bool VEC>
__device__ __forceinline__ v4u load_group(const T* __restrict__ p, int64_t have) {
  constexpr int G = Mma<T>::kGroup;
  if constexpr (VEC) {
    if (have <= 0) return v4u{0, 0, 0, 0};
    return *reinterpret_cast<const v4u*>(p);
  } else {
    uint32_t e[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
      e[k] = 0;
      if (k < have) {
        if constexpr (sizeof(T) == 2) e[k] = p[k]; else e[k] = __float_as_uint(p[k]);
      }
    }
    if constexpr (G == 8) return v4u{e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16)};
    else return v4u{e[0], e[1], e[2], e[3]};
  }
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
// Parts that h is split into for adapters of type T and outputs of type YT.
template <typename T, typename YT>
constexpr int expand_parts() { return sizeof(T) == 4 ? 1 : (sizeof(YT) == 2 ? 2 : 3); }
constexpr int kReduceWaves = 4;

}  // namespace

// ------------------------------------------------------------------------------ reduce ----

// Workgroup: 16 TR rows x one chunk of the contraction x the tile's segments s with s % Q == q; its
// four waves take a quarter of the chunk each and join in LDS.  Output: fp32 partial sums
// part[chunk][row][rp], each (chunk, row) written by exactly one workgroup (the one whose segment
// holds the row); rows without an adapter are not written.  Loads are range-checked buffer loads, all of
// U steps issued before the first product, and U more while those are multiplied.
template <typename T, int RT, int TR, bool VEC>
__global__ __launch_bounds__(64 * kReduceWaves) void k_reduce(LoraReduceGroup grp, const int32_t* __restrict__ seg_start,
                                                              const int32_t* __restrict__ seg_adapter, int S, int L,
                                                              int N, int r, int Q) {
  constexpr int G = Mma<T>::kGroup, kStep = 4 * G;
  constexpr int U = RT * TR > 8 || RT > 4 ? 1 : 2;
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
      if constexpr (VEC) {
        const uint32_t voff = kk < kend ? (uint32_t)((row * K + kk) * sizeof(T)) : kNoLoad;
        o[t] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(rs_x, voff, 0, 0));
      } else {
        o[t] = load_group<T, false>(x + min(row, (int64_t)(t1 - t0 - 1)) * K + kk, kend - kk);
      }
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
#pragma unroll
        for (int u = 0; u < U; ++u) {
          load_x(k + ((h + 1) * U + u) * kStep, xs[h ^ 1][u]);
          load_w(k + ((h + 1) * U + u) * kStep, ws[h ^ 1][u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int v = 0; v < TR; ++v) acc[t][v] = Mma<T>::run(ws[h][u][t], xs[h][u][v], acc[t][v]);
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

// One lane's operand group for k_expand from G sums: part `part` of the bf16 split (hi, then what is
// left, then what is left of that), or the fp32 values.
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
      float v = h[j];
      uint32_t w = f32_to_bf16_rne(v);
      // a part that is not finite carries everything: the later parts are 0, not inf - inf
      for (int p = 0; p < part; ++p) {
        const float hi = __uint_as_float(w << 16);
        v = isfinite(hi) ? v - hi : 0.f;
        w = f32_to_bf16_rne(v);
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

// For each 16-row tile: the chunks' partial sums joined and scaled by the row's alpha, written as
// fp32 rows [N][rp] (item.joined) and / or as k_expand's operand groups [tile][step][lane]
// (item.groups), each optional.  Rows without an adapter give 0.  One wave per tile.
template <typename T>
__global__ __launch_bounds__(256) void k_reduce_join(LoraReduceGroup grp, const int32_t* __restrict__ seg_start,
                                                     const int32_t* __restrict__ seg_adapter, int S, int L, int N,
                                                     int rp, int parts) {
  constexpr int G = Mma<T>::kGroup;
  const LoraReduceItem& it = grp.items[blockIdx.y];
  const int lane = threadIdx.x & (kWave - 1), c = lane & 15;
  const int gpp = rp / G;
  const int steps = (parts * gpp + 3) / 4;
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);   // (tile, step)
  const int tile = unit / steps, st = unit % steps;
  const int t0 = tile * kRows;
  if (t0 >= N) return;
  const int grpi = st * 4 + (lane >> 4), part = grpi / gpp, k = (grpi % gpp) * G, row = t0 + c;
  Segments segs(seg_start, seg_adapter, S, L, t0, min(t0 + kRows, N), 0, 1, lane);
  int own = -1;
  for (int lo, hi, a; segs.next(lo, hi, a);)
    if (row >= lo && row < hi) own = a;
  float v[G];
#pragma unroll
  for (int j = 0; j < G; ++j) v[j] = 0.f;
  if (own >= 0 && part < parts) {
    const float al = it.alpha[own];
    join_chunks<G>(it.part, (int64_t)row * rp + k, (int64_t)N * rp, (int)((it.K + it.chunk - 1) / it.chunk), v);
#pragma unroll
    for (int j = 0; j < G; ++j) v[j] *= al;
  }
  if (it.joined && part == 0 && row < N) {
#pragma unroll
    for (int j = 0; j < G; j += 4)
      *reinterpret_cast<v4f*>(it.joined + (int64_t)row * rp + k + j) = v4f{v[j], v[j + 1], v[j + 2], v[j + 3]};
  }
  if (it.groups) static_cast<v4u*>(it.groups)[((int64_t)tile * steps + st) * 64 + lane] =
      part < parts ? operand_group<T>(v, part) : v4u{0, 0, 0, 0};
}

// ------------------------------------------------------------------------------ expand ----

// Workgroup: 16 TF rows x 256 outputs (64 per wave) x the segments s with s % Q == q; for each segment
// it multiplies and stores base + delta.  The rows' operand groups come from k_reduce_join (READY: long
// segments, where every workgroup of a row tile would join the same sums again) or are made here from
// the partial sums (few rows: one launch less).  base is loaded first of all, so that it arrives while
// the segments, the groups and the adapter do.
//
// Row i of output fragment f of a 64-output group is output 16 (i / 4) + 4 f + i % 4, so that the
// accumulators of a lane over the four fragments are 16 consecutive outputs of one row.
template <typename T, typename YT, int TF, bool READY, bool WVEC>
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
  const int64_t o_block = (int64_t)blockIdx.y * 256, o0 = o_block + wave * 64;
  if (o_block >= M) return;
  const int t0 = (int)(blockIdx.x / Q) * kTile, q = blockIdx.x % Q;
  const int t1 = min(t0 + kTile, N);
  const int gpp = rp / G;                                  // operand groups per part
  const int steps = (kParts * gpp + 3) / 4;
  const YT* base = static_cast<const YT*>(it.base);
  YT* y = static_cast<YT*>(it.y);
  const bool yvec = (M * sizeof(YT)) % 16 == 0 && o0 + 16 * g + 16 <= M;
  v4u old[TF][kBase];
#pragma unroll
  for (int t = 0; t < TF; ++t)
    if (yvec) {
      const int64_t row = min(t0 + 16 * t + c, t1 - 1);
#pragma unroll
      for (int i = 0; i < kBase; ++i)
        old[t][i] = *reinterpret_cast<const v4u*>(base + row * M + o0 + 16 * g + i * (16 / kBase));
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
    for (int st = 0; st < steps; ++st) {
      const int grpi = st * 4 + g, k = (grpi % gpp) * G;
      const int have = grpi < kParts * gpp ? r - k : 0;
      v4u wa[4], hb[TF];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int o = 16 * (c >> 2) + 4 * f + (c & 3);
        if constexpr (WVEC) {
          wa[f] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(
              rs_w, have > 0 ? (uint32_t)((o * r + k) * sizeof(T)) : kNoLoad, 0, 0));
        } else {
          wa[f] = load_group<T, false>(Wa + min((int64_t)o, M - 1 - o0) * r + k, have);
        }
      }
#pragma unroll
      for (int t = 0; t < TF; ++t) hb[t] = groups[(min(t, tiles_here - 1) * steps + st) * 64 + lane];
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t) acc[f][t] = Mma<T>::run(wa[f], hb[t], acc[f][t]);
    }
#pragma unroll
    for (int t = 0; t < TF; ++t) {
      const int row = t0 + 16 * t + c;
      if (row < lo || row >= hi) continue;
      const int64_t off = (int64_t)row * M + o0 + 16 * g;
      if (yvec) {
        if constexpr (sizeof(YT) == 4) {
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const v4f b = __builtin_bit_cast(v4f, old[t][f]);
            *reinterpret_cast<v4f*>(y + off + 4 * f) =
                v4f{b[0] + acc[f][t][0], b[1] + acc[f][t][1], b[2] + acc[f][t][2], b[3] + acc[f][t][3]};
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v4u o;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const v4f& d = acc[2 * h + (w >> 1)][t];
              const int e = 2 * (w & 1);
              o[w] = (uint32_t)f32_to_bf16_rne(bf16_lo(old[t][h][w]) + d[e]) |
                     ((uint32_t)f32_to_bf16_rne(bf16_hi(old[t][h][w]) + d[e + 1]) << 16);
            }
            *reinterpret_cast<v4u*>(y + off + 8 * h) = o;
          }
        }
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (o0 + 16 * g + 4 * f + e < M) {
              const int64_t i = off + 4 * f + e;
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
// in [L][R][C] -> out [L][C][ldo], columns R..ldo-1 zeroed.  blockIdx.y picks the matrix.
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

// dA (dB): for adapter a, columns of x (dy) and 16 ranks, the sum over the adapter's rows of
// factor[row][rank] * x[row][col], all fp32.  Workgroup: 128 columns (two per lane) x 16 ranks x the
// rows [split * span, (split + 1) * span); its four waves take every fourth row and join in LDS in
// wave order.  The factor is wave-uniform: it arrives over scalar loads.  Splits are joined in order
// by k_outer_join (splits > 1), so the result never depends on scheduling.
template <typename T>
__global__ __launch_bounds__(256) void k_outer(LoraOuterGroup grp, const int32_t* __restrict__ seg_start,
                                               const int32_t* __restrict__ seg_adapter, int S, int L, int N, int r,
                                               int rp, int splits, int span) {
  __shared__ float s_sum[4][128][17];
  const int half = blockIdx.z & 1;
  const LoraOuterItem& it = grp.items[half];
  const int a = (int)(blockIdx.z >> 1);
  const int64_t C = it.C;
  const int64_t c0 = (int64_t)blockIdx.x * 128;
  if (c0 >= C) return;
  const int rt = blockIdx.y / splits, split = blockIdx.y % splits;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int t0 = split * span, t1 = min(t0 + span, N);
  const T* __restrict__ x = static_cast<const T*>(it.x);
  const float* __restrict__ fac = it.factor + rt * 16;
  const T* __restrict__ xc = x + min(c0 + 2 * lane, C - 2);      // C is even: a pair never straddles the end
  constexpr int kDeep = 4;                                 // rows whose loads are in flight together
  float acc[2][16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[0][k] = acc[1][k] = 0.f;
  Segments segs(seg_start, seg_adapter, S, L, t0, t1, 0, 1, lane);
  int lo, hi, who;
  while (segs.next(lo, hi, who)) {
    if (who != a) continue;
    for (int row0 = lo + wave; row0 < hi; row0 += 4 * kDeep) {
      float v[kDeep][2];
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {                    // rows past the segment repeat its last one
        const int64_t row = min(row0 + 4 * d, hi - 1);
        if constexpr (sizeof(T) == 4) {
          const float2 w = *reinterpret_cast<const float2*>(xc + row * C);
          v[d][0] = w.x;
          v[d][1] = w.y;
        } else {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(xc + row * C);
          v[d][0] = bf16_lo(w);
          v[d][1] = bf16_hi(w);
        }
      }
#pragma unroll
      for (int d = 0; d < kDeep; ++d) {
        if (row0 + 4 * d >= hi) break;
        const float* __restrict__ f = fac + (int64_t)(row0 + 4 * d) * rp;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          acc[0][k] = fmaf(v[d][0], f[k], acc[0][k]);
          acc[1][k] = fmaf(v[d][1], f[k], acc[1][k]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    s_sum[wave][2 * lane][k] = acc[0][k];
    s_sum[wave][2 * lane + 1][k] = acc[1][k];
  }
  __syncthreads();
  float* __restrict__ out = it.out + ((int64_t)split * L + a) * r * C;
  for (int e = threadIdx.x; e < 128 * 16; e += 256) {
    const int col = it.rank_major ? e % 128 : e / 16, k = it.rank_major ? e / 128 : e % 16;
    const int rank = rt * 16 + k;
    if (c0 + col >= C || rank >= r) continue;
    const float v = ((s_sum[0][col][k] + s_sum[1][col][k]) + s_sum[2][col][k]) + s_sum[3][col][k];
    out[it.rank_major ? (int64_t)rank * C + c0 + col : (c0 + col) * r + rank] = v;
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
// of x, so long segments take 64 rows to one read of it.
int reduce_rows(int N, int S, int r) { return segment_shares(N, S) == 1 && N >= 256 && r > 32 ? 4 : 1; }

// Contraction chunk of k_reduce: small enough that the launch has about 2048 workgroups, at least
// 256 elements (each wave then runs two bf16 steps), a multiple of 256.
int reduce_chunk(int64_t K, int N, int S, int r, int items) {
  const int tile = kRows * reduce_rows(N, S, r);
  const int64_t wgs = (int64_t)((N + tile - 1) / tile) * segment_shares(N, S) * items;
  const int64_t want = std::max<int64_t>(1, 2048 / wgs);
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
  const dim3 grid((N + tile - 1) / tile * Q, most, count);
  switch (rank_tiles(r)) {
    case 1: reduce_vec<T, 1, 1>(grp, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    case 2: reduce_vec<T, 2, 1>(grp, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    case 4:
      if (tr == 4) reduce_vec<T, 4, 4>(grp, vec, grid, ss, sa, S, L, N, r, Q, st);
      else reduce_vec<T, 4, 1>(grp, vec, grid, ss, sa, S, L, N, r, Q, st);
      break;
    default:
      if (tr == 4) reduce_vec<T, 8, 4>(grp, vec, grid, ss, sa, S, L, N, r, Q, st);
      else reduce_vec<T, 8, 1>(grp, vec, grid, ss, sa, S, L, N, r, Q, st);
      break;
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
  if (r % Mma<T>::kGroup == 0)
    hipLaunchKernelGGL((k_expand<T, YT, TF, READY, true>), grid, dim3(256), lds, st, grp, ss, sa, S, L, N, r, rp, Q);
  else
    hipLaunchKernelGGL((k_expand<T, YT, TF, READY, false>), grid, dim3(256), lds, st, grp, ss, sa, S, L, N, r, rp, Q);
}

// Rows per workgroup of k_expand: 16 for few rows or short segments, 32 otherwise (an adapter fragment
// then serves two row tiles, and four waves a SIMD still fit).
template <typename T, typename YT>
void launch_expand(const LoraExpandGroup& grp, int count, const int32_t* ss, const int32_t* sa, int S, int L, int N,
                   int r, hipStream_t st) {
  if (ready_groups(N, S)) expand_tf<T, YT, 2, true>(grp, count, ss, sa, S, L, N, r, 1, st);
  else expand_tf<T, YT, 1, false>(grp, count, ss, sa, S, L, N, r, segment_shares(N, S), st);
}

template <typename T>
void launch_expand_y(const LoraExpandGroup& grp, int count, int y_bf16, const int32_t* ss, const int32_t* sa, int S,
                     int L, int N, int r, hipStream_t st) {
  if (y_bf16) launch_expand<T, uint16_t>(grp, count, ss, sa, S, L, N, r, st);
  else launch_expand<T, float>(grp, count, ss, sa, S, L, N, r, st);
}

template <typename T>
void launch_join(const LoraReduceGroup& grp, int count, int y_bf16, const int32_t* ss, const int32_t* sa, int S, int L,
                 int N, int r, hipStream_t st) {
  const int units = (N + kRows - 1) / kRows * group_steps(r, sizeof(T), y_bf16);
  hipLaunchKernelGGL((k_reduce_join<T>), dim3((units + 3) / 4, count), dim3(256), 0, st, grp, ss, sa, S, L, N,
                     16 * rank_tiles(r), sizeof(T) == 4 ? 1 : (y_bf16 ? 2 : 3));
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

size_t lora_part_floats(int64_t K, int chunk, int64_t N, int r) { return (size_t)chunks(K, chunk) * N * 16 * rank_tiles(r); }

template <typename T>
hipError_t lora_t(const LoraArgs& p, const LoraItem* items, int count, hipStream_t st) {
  const int64_t K = 2 * p.m;
  const int chunk = reduce_chunk(K, p.N, p.S, p.r, count);
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
  if (ready) launch_join<T>(red, count, p.y_bf16, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_expand_y<T>(exp, count, p.y_bf16, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  return hipGetLastError();
}

// Row ranges of k_outer: enough workgroups for the device when there are few adapters and columns,
// at least 64 rows each.
int outer_splits(int64_t N, int64_t C, int r, int L) {
  const int64_t wgs = (C + 127) / 128 * ((r + 15) / 16) * L * 2;
  const int64_t want = std::max<int64_t>(1, 1024 / wgs);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, N / 64));
}

struct BackwardPlan {
  int rp, chunk_x, chunk_y, splits, span;
  int64_t K, M, Mp;
  size_t part_x, part_y, joined, groups, bt, at, outer_a, outer_b, total;
};

BackwardPlan backward_plan(int64_t N, int64_t m, int64_t n, int r, int L, int S, int elem) {
  BackwardPlan b;
  b.rp = 16 * rank_tiles(r);
  b.K = 2 * m;
  b.M = 2 * n;
  b.Mp = (b.M + 63) / 64 * 64;
  b.chunk_x = reduce_chunk(b.K, (int)N, S, r, 2);
  b.chunk_y = reduce_chunk(b.M, (int)N, S, r, 2);
  b.splits = outer_splits(N, std::max(b.K, b.M), r, L);
  b.span = (int)((N + b.splits - 1) / b.splits);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
  b.part_x = take((size_t)chunks(b.K, b.chunk_x) * N * b.rp * 4);
  b.part_y = take((size_t)chunks(b.M, b.chunk_y) * N * b.rp * 4);
  b.joined = take((size_t)2 * N * b.rp * 4);
  b.groups = take(group_bytes(N, r, elem, 0));           // an fp32 dx has the most parts
  b.bt = take((size_t)L * r * b.Mp * elem);
  b.at = take((size_t)L * b.K * r * elem);
  b.outer_a = take(b.splits > 1 ? (size_t)b.splits * L * r * b.K * 4 : 0);
  b.outer_b = take(b.splits > 1 ? (size_t)b.splits * L * r * b.M * 4 : 0);
  b.total = at;
  return b;
}

template <typename T>
hipError_t lora_backward_t(const LoraBackwardArgs& p, hipStream_t st) {
  const BackwardPlan b = backward_plan(p.N, p.m, p.n, p.r, p.L, p.S, sizeof(T));
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  float* h = reinterpret_cast<float*>(ws + b.joined);
  float* dh = h + (size_t)p.N * b.rp;
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
  red.items[0] = LoraReduceItem{p.x, p.A, reinterpret_cast<float*>(ws + b.part_x), h, nullptr, p.alpha, b.K, b.K, b.chunk_x};
  red.items[1] = LoraReduceItem{p.dy, Bt, part_y, dh, p.dx && ready ? ws + b.groups : nullptr, p.alpha, b.M, b.Mp, b.chunk_y};
  launch_reduce<T>(red, 2, vec, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  launch_join<T>(red, 2, p.dx_bf16, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  if (p.dx) {
    LoraExpandGroup exp;
    exp.items[0] = LoraExpandItem{part_y, ws + b.groups, At, p.alpha, p.dx_base, p.dx, b.K, chunks(b.M, b.chunk_y)};
    launch_expand_y<T>(exp, 1, p.dx_bf16, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  }
  LoraOuterGroup out;
  float* da = b.splits > 1 ? reinterpret_cast<float*>(ws + b.outer_a) : p.dA;
  float* db = b.splits > 1 ? reinterpret_cast<float*>(ws + b.outer_b) : p.dB;
  out.items[0] = LoraOuterItem{p.x, dh, da, b.K, 1};
  out.items[1] = LoraOuterItem{p.dy, h, db, b.M, 0};
  hipLaunchKernelGGL((k_outer<T>), dim3((unsigned)((std::max(b.K, b.M) + 127) / 128), (p.r + 15) / 16 * b.splits, 2 * p.L),
                     block, 0, st, out, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, b.rp, b.splits, b.span);
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
    const int chunk = reduce_chunk(2 * m, (int)N, (int)S, r, items);
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
