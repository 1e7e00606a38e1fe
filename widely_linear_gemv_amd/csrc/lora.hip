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

// First segment whose end lies past row `row` (S if none); seg_start is nondecreasing.  Every lane
// of the wave calls it and gets the same answer: 64 offsets are compared at a time.
__device__ __forceinline__ int first_segment(const int32_t* __restrict__ seg_start, int S, int row, int lane) {
  for (int s0 = 0; s0 < S; s0 += kWave) {
    const int s = s0 + lane;
    const uint64_t past = __ballot(s < S && seg_start[min(s, S - 1) + 1] > row);
    if (past) return s0 + __builtin_ctzll(past);
  }
  return S;
}

// Adapter of a segment, -1 if it has none.
__device__ __forceinline__ int adapter_of(const int32_t* __restrict__ seg_adapter, int s, int L) {
  const int a = seg_adapter[s];
  return a >= 0 && a < L ? a : -1;
}

constexpr int kRows = 16;              // rows of x per tile
constexpr int kReduceWaves = 4;

}  // namespace

// ------------------------------------------------------------------------------ reduce ----

// Workgroup: 16 rows x one chunk of the contraction x the tile's segments s with s % Q == q; its
// four waves take a quarter of the chunk each and join in LDS.  Output: fp32 partial sums
// part[chunk][row][rp], each (chunk, row) written by exactly one workgroup (the one whose segment
// holds the row); rows without an adapter are not written.
template <typename T, int RT, bool VEC>
__global__ __launch_bounds__(64 * kReduceWaves) void k_reduce(LoraReduceGroup grp, const int32_t* __restrict__ seg_start,
                                                              const int32_t* __restrict__ seg_adapter, int S, int L,
                                                              int N, int r, int Q) {
  constexpr int G = Mma<T>::kGroup, kStep = 4 * G;
  __shared__ __align__(16) float s_part[kReduceWaves][kRows][RT * 16];
  const LoraReduceItem& it = grp.items[blockIdx.z];
  const int chunk = blockIdx.y;
  if ((int64_t)chunk * it.chunk >= it.K) return;
  const T* __restrict__ x = static_cast<const T*>(it.x);
  const T* __restrict__ W = static_cast<const T*>(it.W);
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = (int)(blockIdx.x / Q) * kRows, q = blockIdx.x % Q;
  const int t1 = min(t0 + kRows, N);
  const int rp = RT * 16;
  const int64_t K = it.K;
  const int per_wave = it.chunk / kReduceWaves;
  const int64_t k0 = (int64_t)chunk * it.chunk + (int64_t)wave * per_wave;
  const int64_t kend = min(k0 + per_wave, K);
  const T* __restrict__ xr = x + (int64_t)min(t0 + c, N - 1) * K;

  for (int s = first_segment(seg_start, S, t0, lane); s < S; ++s) {
    const int lo = max(seg_start[s], t0), hi = min(seg_start[s + 1], t1);
    if (seg_start[s] >= t1) break;
    if (s % Q != q || lo >= hi) continue;
    const int a = adapter_of(seg_adapter, s, L);
    if (a < 0) continue;
    const T* __restrict__ Wa = W + (int64_t)a * r * it.ldw;
    v4f acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int64_t k = k0; k < kend; k += kStep) {
      const int64_t kk = k + g * G;
      const v4u xb = load_group<T, VEC>(xr + kk, K - kk);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const v4u wa = load_group<T, true>(Wa + (int64_t)min(t * 16 + c, r - 1) * it.ldw + kk, K - kk);
        acc[t] = Mma<T>::run(wa, xb, acc[t]);
      }
    }
    // C: lane holds ranks 16 t + 4 g .. + 3 of row c
#pragma unroll
    for (int t = 0; t < RT; ++t) *reinterpret_cast<v4f*>(&s_part[wave][c][t * 16 + 4 * g]) = acc[t];
    __syncthreads();
    for (int e = threadIdx.x; e < kRows * rp; e += 64 * kReduceWaves) {
      const int row = t0 + e / rp, k = e % rp;
      if (row >= lo && row < hi && k < r) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kReduceWaves; ++w) v += s_part[w][row - t0][k];
        it.part[((int64_t)chunk * N + row) * rp + k] = v;
      }
    }
    __syncthreads();
  }
}

// Joins the chunks' partial sums in order and scales them by the row's alpha: out [N][rp], zeros in
// ranks r..rp-1 and in rows without an adapter.
__global__ __launch_bounds__(256) void k_reduce_join(LoraReduceGroup grp, const float* __restrict__ alpha,
                                                     const int32_t* __restrict__ seg_start,
                                                     const int32_t* __restrict__ seg_adapter, int S, int L, int N,
                                                     int r, int rp) {
  const LoraReduceItem& it = grp.items[blockIdx.y];
  const int lane = threadIdx.x & (kWave - 1);
  const int per = 256 / 64;                                   // one row per wave and pass
  const int row = blockIdx.x * per + threadIdx.x / kWave;
  if (row >= N) return;
  const int s = first_segment(seg_start, S, row, lane);
  const int a = s < S && seg_start[s] <= row ? adapter_of(seg_adapter, s, L) : -1;
  const int nchunk = (int)((it.K + it.chunk - 1) / it.chunk);
  for (int k = lane; k < rp; k += kWave) {
    float v = 0.f;
    if (a >= 0 && k < r) {
      for (int ch = 0; ch < nchunk; ++ch) v += it.part[((int64_t)ch * N + row) * rp + k];
      v *= alpha[a];
    }
    it.joined[(int64_t)row * rp + k] = v;
  }
}

// ------------------------------------------------------------------------------ expand ----

// Workgroup: 16 TF rows x 256 outputs (64 per wave) x the segments s with s % Q == q.  It first joins
// its rows' partial sums (h, scaled by alpha unless the partials are scaled already) into LDS and
// splits them into operand groups; then for each segment multiplies and stores base + delta.
//
// Row i of output fragment f of a 64-output group is output 16 (i / 4) + 4 f + i % 4, so that the
// accumulators of a lane over the four fragments are 16 consecutive outputs of one row.
template <typename T, typename YT, int TF, bool WVEC>
__global__ __launch_bounds__(256) void k_expand(LoraExpandGroup grp, const int32_t* __restrict__ seg_start,
                                                const int32_t* __restrict__ seg_adapter, int S, int L, int N, int r,
                                                int rp, int Q) {
  constexpr int G = Mma<T>::kGroup;
  constexpr int kParts = sizeof(T) == 4 ? 1 : (sizeof(YT) == 2 ? 2 : 3);
  constexpr int kTile = kRows * TF;
  extern __shared__ __align__(16) uint8_t s_mem[];
  const LoraExpandItem& it = grp.items[blockIdx.z];
  const int64_t M = it.M;
  const int o_block = blockIdx.y * 256;
  if (o_block >= M) return;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = (int)(blockIdx.x / Q) * kTile, q = blockIdx.x % Q;
  const int t1 = min(t0 + kTile, N);
  const int gpp = rp / G;                                  // operand groups per part
  const int steps = (kParts * gpp + 3) / 4;
  float* s_h = reinterpret_cast<float*>(s_mem);            // [kTile][rp]
  v4u* s_frag = reinterpret_cast<v4u*>(s_mem + (size_t)kTile * rp * 4);   // [steps][TF][64]

  const int first = first_segment(seg_start, S, t0, lane);
  for (int e = threadIdx.x; e < kTile * rp; e += 256) s_h[e] = 0.f;
  __syncthreads();
  for (int s = first; s < S && seg_start[s] < t1; ++s) {
    const int lo = max(seg_start[s], t0), hi = min(seg_start[s + 1], t1);
    if (s % Q != q || lo >= hi) continue;
    const int a = adapter_of(seg_adapter, s, L);
    if (a < 0) continue;
    const float al = it.alpha ? it.alpha[a] : 1.f;
    for (int e = threadIdx.x; e < (hi - lo) * rp; e += 256) {
      const int row = lo + e / rp, k = e % rp;
      if (k >= r) continue;
      float v = 0.f;
      for (int ch = 0; ch < it.nchunk; ++ch) v += it.part[((int64_t)ch * N + row) * rp + k];
      s_h[(row - t0) * rp + k] = v * al;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < steps * TF * 64; e += 256) {
    const int st = e / (TF * 64), f = (e / 64) % TF, l = e % 64;
    const int grpi = st * 4 + (l >> 4), part = grpi / gpp, k = (grpi % gpp) * G, row = f * 16 + (l & 15);
    v4u o = v4u{0, 0, 0, 0};
    if (part < kParts) {
      if constexpr (sizeof(T) == 4) {
        o = *reinterpret_cast<const v4u*>(&s_h[row * rp + k]);
      } else {
        uint32_t b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = s_h[row * rp + k + j];
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
    }
    s_frag[e] = o;
  }
  __syncthreads();

  const int o0 = o_block + wave * 64;
  if (o0 >= M) return;
  const T* __restrict__ W = static_cast<const T*>(it.W);
  const YT* base = static_cast<const YT*>(it.base);
  YT* y = static_cast<YT*>(it.y);
  const bool yvec = (M * sizeof(YT)) % 16 == 0 && o0 + 16 * g + 16 <= M;
  for (int s = first; s < S && seg_start[s] < t1; ++s) {
    const int lo = max(seg_start[s], t0), hi = min(seg_start[s + 1], t1);
    if (s % Q != q || lo >= hi) continue;
    const int a = adapter_of(seg_adapter, s, L);
    if (a < 0) continue;
    const T* __restrict__ Wa = W + (int64_t)a * M * r;
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
        const int64_t o = min((int64_t)(o0 + 16 * (c >> 2) + 4 * f + (c & 3)), M - 1);
        wa[f] = load_group<T, WVEC>(Wa + o * r + k, have);
      }
#pragma unroll
      for (int t = 0; t < TF; ++t) hb[t] = s_frag[(st * TF + t) * 64 + lane];
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
            const v4f b = *reinterpret_cast<const v4f*>(base + off + 4 * f);
            *reinterpret_cast<v4f*>(y + off + 4 * f) =
                v4f{b[0] + acc[f][t][0], b[1] + acc[f][t][1], b[2] + acc[f][t][2], b[3] + acc[f][t][3]};
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4u b = *reinterpret_cast<const v4u*>(base + off + 8 * h);
            v4u o;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const v4f& d = acc[2 * h + (w >> 1)][t];
              const int e = 2 * (w & 1);
              o[w] = (uint32_t)f32_to_bf16_rne(bf16_lo(b[w]) + d[e]) |
                     ((uint32_t)f32_to_bf16_rne(bf16_hi(b[w]) + d[e + 1]) << 16);
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
// in [L][R][C] -> out [L][C][ldo], columns R..ldo-1 zeroed (ldo a multiple of 16 bytes' elements).
template <typename T>
__global__ __launch_bounds__(256) void k_transpose(const T* __restrict__ in, T* __restrict__ out, int64_t R, int64_t C,
                                                   int64_t ldo) {
  __shared__ T s[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c0 = (int64_t)blockIdx.x * 32, r0 = (int64_t)blockIdx.y * 32;
  in += (int64_t)blockIdx.z * R * C;
  out += (int64_t)blockIdx.z * C * ldo;
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    const int64_t rr = r0 + ty + j, cc = c0 + tx;
    s[ty + j][tx] = rr < R && cc < C ? in[rr * C + cc] : T(0);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    const int64_t cc = c0 + ty + j, rr = r0 + tx;
    if (cc < C && rr < ldo) out[cc * ldo + rr] = s[tx][ty + j];
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
  const int64_t ca = min(c0 + 2 * lane, C - 1), cb = min(c0 + 2 * lane + 1, C - 1);
  float acc[2][16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[0][k] = acc[1][k] = 0.f;
  for (int s = first_segment(seg_start, S, t0, lane); s < S && seg_start[s] < t1; ++s) {
    if (seg_adapter[s] != a) continue;
    const int lo = max(seg_start[s], t0), hi = min(seg_start[s + 1], t1);
    for (int row = lo + wave; row < hi; row += 4) {
      float v0, v1;
      if constexpr (sizeof(T) == 4) {
        v0 = x[row * C + ca];
        v1 = x[row * C + cb];
      } else {
        v0 = bf16_lo(x[row * C + ca]);
        v1 = bf16_lo(x[row * C + cb]);
      }
      const float* __restrict__ f = fac + (int64_t)row * rp;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        acc[0][k] = fmaf(v0, f[k], acc[0][k]);
        acc[1][k] = fmaf(v1, f[k], acc[1][k]);
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

__global__ __launch_bounds__(256) void k_outer_join(const float* __restrict__ part, float* __restrict__ out, int64_t n,
                                                    int splits) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = part[i];
  for (int s = 1; s < splits; ++s) v += part[(int64_t)s * n + i];
  out[i] = v;
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

// Contraction chunk of k_reduce: small enough that the launch has about 512 workgroups, at least
// 256 elements (each wave then runs two bf16 steps), a multiple of 256.
int reduce_chunk(int64_t K, int N, int S, int items) {
  const int64_t wgs = (int64_t)((N + kRows - 1) / kRows) * segment_shares(N, S) * items;
  const int64_t want = std::max<int64_t>(1, 512 / wgs);
  const int64_t chunk = (K + want - 1) / want;
  return (int)std::max<int64_t>(256, (chunk + 255) / 256 * 256);
}

int chunks(int64_t K, int chunk) { return (int)((K + chunk - 1) / chunk); }

template <typename T, int RT>
void reduce_vec(const LoraReduceGroup& grp, int count, bool vec, dim3 grid, const int32_t* ss, const int32_t* sa, int S,
                int L, int N, int r, int Q, hipStream_t st) {
  grid.z = count;
  if (vec) hipLaunchKernelGGL((k_reduce<T, RT, true>), grid, dim3(64 * kReduceWaves), 0, st, grp, ss, sa, S, L, N, r, Q);
  else hipLaunchKernelGGL((k_reduce<T, RT, false>), grid, dim3(64 * kReduceWaves), 0, st, grp, ss, sa, S, L, N, r, Q);
}

template <typename T>
void launch_reduce(const LoraReduceGroup& grp, int count, bool vec, const int32_t* ss, const int32_t* sa, int S, int L,
                   int N, int r, hipStream_t st) {
  const int Q = segment_shares(N, S);
  int most = 1;
  for (int k = 0; k < count; ++k) most = std::max(most, chunks(grp.items[k].K, grp.items[k].chunk));
  const dim3 grid((N + kRows - 1) / kRows * Q, most, count);
  switch (rank_tiles(r)) {
    case 1: reduce_vec<T, 1>(grp, count, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    case 2: reduce_vec<T, 2>(grp, count, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    case 4: reduce_vec<T, 4>(grp, count, vec, grid, ss, sa, S, L, N, r, Q, st); break;
    default: reduce_vec<T, 8>(grp, count, vec, grid, ss, sa, S, L, N, r, Q, st); break;
  }
}

template <typename T, typename YT, int TF>
void expand_tf(const LoraExpandGroup& grp, int count, const int32_t* ss, const int32_t* sa, int S, int L, int N, int r,
               int Q, hipStream_t st) {
  const int rp = 16 * rank_tiles(r);
  constexpr int G = Mma<T>::kGroup, kParts = sizeof(T) == 4 ? 1 : (sizeof(YT) == 2 ? 2 : 3);
  const int steps = (kParts * (rp / G) + 3) / 4;
  const size_t lds = (size_t)kRows * TF * rp * 4 + (size_t)steps * TF * 64 * 16;
  int64_t most = 0;
  for (int k = 0; k < count; ++k) most = std::max(most, grp.items[k].M);
  const int tile = kRows * TF;
  const dim3 grid((N + tile - 1) / tile * Q, (unsigned)((most + 255) / 256), count);
  const bool wvec = r % G == 0;
  if (wvec) hipLaunchKernelGGL((k_expand<T, YT, TF, true>), grid, dim3(256), lds, st, grp, ss, sa, S, L, N, r, rp, Q);
  else hipLaunchKernelGGL((k_expand<T, YT, TF, false>), grid, dim3(256), lds, st, grp, ss, sa, S, L, N, r, rp, Q);
}

// Rows per workgroup of k_expand: 16 for short segments (Q > 1) or few rows, 64 otherwise (an
// adapter fragment then serves four row tiles).
template <typename T, typename YT>
void launch_expand(const LoraExpandGroup& grp, int count, const int32_t* ss, const int32_t* sa, int S, int L, int N,
                   int r, hipStream_t st) {
  const int Q = segment_shares(N, S);
  if (Q > 1 || N <= 64) expand_tf<T, YT, 1>(grp, count, ss, sa, S, L, N, r, Q, st);
  else expand_tf<T, YT, 4>(grp, count, ss, sa, S, L, N, r, 1, st);
}

template <typename T>
void launch_expand_y(const LoraExpandGroup& grp, int count, int y_bf16, const int32_t* ss, const int32_t* sa, int S,
                     int L, int N, int r, hipStream_t st) {
  if (y_bf16) launch_expand<T, uint16_t>(grp, count, ss, sa, S, L, N, r, st);
  else launch_expand<T, float>(grp, count, ss, sa, S, L, N, r, st);
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

template <typename T>
hipError_t lora_t(const LoraArgs& p, const LoraItem* items, int count, hipStream_t st) {
  const int rp = 16 * rank_tiles(p.r);
  const int64_t K = 2 * p.m;
  const int chunk = reduce_chunk(K, p.N, p.S, count);
  const size_t part = (size_t)chunks(K, chunk) * p.N * rp;
  LoraReduceGroup red;
  LoraExpandGroup exp;
  for (int k = 0; k < count; ++k) {
    float* w = static_cast<float*>(p.ws) + part * k;
    red.items[k] = LoraReduceItem{p.x, items[k].A, w, nullptr, K, K, chunk};
    exp.items[k] = LoraExpandItem{w, items[k].B, items[k].alpha, items[k].base, items[k].y, 2 * items[k].n,
                                  chunks(K, chunk)};
  }
  launch_reduce<T>(red, count, true, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  hipError_t e = hipGetLastError();
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
  size_t part_x, part_y, joined, bt, at, outer_a, outer_b, total;
};

BackwardPlan backward_plan(int64_t N, int64_t m, int64_t n, int r, int L, int S, int elem) {
  BackwardPlan b;
  b.rp = 16 * rank_tiles(r);
  b.K = 2 * m;
  b.M = 2 * n;
  b.Mp = (b.M + 63) / 64 * 64;
  b.chunk_x = reduce_chunk(b.K, (int)N, S, 2);
  b.chunk_y = reduce_chunk(b.M, (int)N, S, 2);
  b.splits = outer_splits(N, std::max(b.K, b.M), r, L);
  b.span = (int)((N + b.splits - 1) / b.splits);
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
  b.part_x = take((size_t)chunks(b.K, b.chunk_x) * N * b.rp * 4);
  b.part_y = take((size_t)chunks(b.M, b.chunk_y) * N * b.rp * 4);
  b.joined = take((size_t)2 * N * b.rp * 4);
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
  hipLaunchKernelGGL((k_transpose<T>), dim3((p.r + 31) / 32, (unsigned)((b.Mp + 31) / 32), p.L), block, 0, st,
                     static_cast<const T*>(p.B), Bt, b.M, (int64_t)p.r, b.Mp);
  if (p.dx)
    hipLaunchKernelGGL((k_transpose<T>), dim3((unsigned)((b.K + 31) / 32), (p.r + 31) / 32, p.L), block, 0, st,
                       static_cast<const T*>(p.A), At, (int64_t)p.r, b.K, (int64_t)p.r);
  const bool vec = (b.M * sizeof(T)) % 16 == 0;
  LoraReduceGroup red;
  red.items[0] = LoraReduceItem{p.x, p.A, reinterpret_cast<float*>(ws + b.part_x), h, b.K, b.K, b.chunk_x};
  red.items[1] = LoraReduceItem{p.dy, Bt, reinterpret_cast<float*>(ws + b.part_y), dh, b.M, b.Mp, b.chunk_y};
  launch_reduce<T>(red, 2, vec, p.seg_start, p.seg_adapter, p.S, p.L, p.N, p.r, st);
  hipLaunchKernelGGL(k_reduce_join, dim3((p.N + 3) / 4, 2), block, 0, st, red, p.alpha, p.seg_start, p.seg_adapter,
                     p.S, p.L, p.N, p.r, b.rp);
  if (p.dx) {
    LoraExpandGroup exp;
    exp.items[0] = LoraExpandItem{dh, At, nullptr, p.dx_base, p.dx, b.K, 1};
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
    hipLaunchKernelGGL(k_outer_join, dim3((unsigned)((na + 255) / 256)), block, 0, st, da, p.dA, na, b.splits);
    hipLaunchKernelGGL(k_outer_join, dim3((unsigned)((nb + 255) / 256)), block, 0, st, db, p.dB, nb, b.splits);
  }
  return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int count, int64_t N, int64_t m, int r, int64_t S) {
  const int per = std::min(count, kMaxLoraItems);
  const int rp = 16 * rank_tiles(r);
  size_t most = 0;
  for (int items : {per, count % kMaxLoraItems}) {
    if (items < 1) continue;
    const int chunk = reduce_chunk(2 * m, (int)N, (int)S, items);
    most = std::max(most, (size_t)items * chunks(2 * m, chunk) * N * rp * 4);
  }
  return up256(most);
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
