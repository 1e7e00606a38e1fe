// Global gradient norm over many tensors, and clipping:
//     norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c g.
//
// Squares and sums are fp64 (the vector ALUs do far more fp64 adds per second than HBM delivers
// values), so no gradient is large or small enough to over- or underflow the sum.  Three passes:
// k_square writes one partial sum per 8192-element piece, k_norm joins them in a fixed order (the
// result never depends on scheduling) into the norm and c, k_scale multiplies.  The norm must be
// known before the first write, so the gradients are read twice; the second time they come from
// the Infinity Cache as far as they fit.  In place with c = 1 nothing is written.
// Bound by memory: 448 fp32 tensors of 44032 to 88064 elements (145 MB) take k_square 44 us (3.3 TB/s; a
// library sum over 1 GiB reads 3.9) and k_scale 48 us (6.0 TB/s read and written, part of it from the
// Infinity Cache).
#include <algorithm>

#include "tiles.hpp"

namespace f2i {

namespace {

constexpr int kPiece = 8192;       // elements per workgroup

// Piece `piece` among all: the last tensor whose first piece is at or before it (64 entries of the table
// are compared at a time), its first element and its elements.
struct Piece {
  const void* g;
  void* out;
  int64_t i0;
  int n;
  bool bf16, vec;
};
__device__ __forceinline__ Piece find_piece(const ClipItem* __restrict__ table, int count, int64_t pieces, int64_t piece) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, len = count;
  while (len > 1) {
    const int stride = (len + kWave - 1) / kWave;
    const int at = lo + lane * stride;
    const uint64_t before = __ballot(at < lo + len && table[min(at, count - 1)].first_piece <= piece);
    const int k = 63 - __builtin_clzll(before | 1);
    lo += k * stride;
    len = min(stride, len - k * stride);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const ClipItem it = table[lo];
  const int64_t last = (lo + 1 < count ? table[lo + 1].first_piece : pieces) - 1;
  return Piece{it.g, it.out, (piece - it.first_piece) * kPiece, piece == last ? (int)it.tail : kPiece,
               (it.flags & kClipBf16) != 0, (it.flags & kClipVec) != 0};
}

__device__ __forceinline__ double sq(float v) { return (double)v * (double)v; }

// Sum over the workgroup in a fixed order; the total is valid in thread 0.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double* s_wave) {
  v = wave_sum(v);
  if ((threadIdx.x & (kWave - 1)) == 0) s_wave[threadIdx.x / kWave] = v;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < THREADS / kWave; ++w) t += s_wave[w];
  return t;
}

}  // namespace

// The table of tensors comes in the kernel arguments, 120 entries to a launch, and is kept in the
// workspace: the passes over the data then run as one launch each, and their thousands of workgroups
// read it from the L2 (arguments lie in host memory: reading the table there took longer than the data).
__global__ __launch_bounds__(64) void k_table(ClipGroup grp, ClipItem* __restrict__ table) {
  for (int k = threadIdx.x; k < grp.count; k += 64) table[k] = grp.items[k];
}

// The 16-byte pieces of an aligned tensor's piece, kPiece / 256 elements to a thread: every load is issued
// before the first is used; elements past the last whole 16 bytes (all, where the tensor is not aligned)
// go one by one.
template <typename T>
struct Chunk {
  static constexpr int kEach = 16 / sizeof(T), kLoads = kPiece / (256 * kEach);
  uint4 w[kLoads];
  int whole;
  __device__ __forceinline__ void load(const T* p, int n, bool vec) {
    whole = vec ? n / kEach * kEach : 0;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = j * 256 + threadIdx.x;
      w[j] = i * kEach < whole ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0, 0, 0, 0);
    }
  }
};
__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(uint16_t v) { return bf16_lo(v); }

template <typename T>
__device__ __forceinline__ double squares(const T* __restrict__ p, int n, bool vec) {
  Chunk<T> q;
  q.load(p, n, vec);
  double v = 0.0;
#pragma unroll
  for (int j = 0; j < Chunk<T>::kLoads; ++j) {
    const uint32_t e[4] = {q.w[j].x, q.w[j].y, q.w[j].z, q.w[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) v += sq(__uint_as_float(e[i]));
      else v += sq(bf16_lo(e[i])) + sq(bf16_hi(e[i]));
    }
  }
#pragma unroll 4
  for (int i = q.whole + threadIdx.x; i < n; i += 256) v += sq(value(p[i]));
  return v;
}

__global__ __launch_bounds__(256) void k_square(const ClipItem* __restrict__ table, int count, int64_t pieces,
                                                int64_t piece0, double* __restrict__ part) {
  __shared__ double s_wave[4];
  const Piece q = find_piece(table, count, pieces, piece0 + blockIdx.x);
  const double v = q.bf16 ? squares(static_cast<const uint16_t*>(q.g) + q.i0, q.n, q.vec)
                          : squares(static_cast<const float*>(q.g) + q.i0, q.n, q.vec);
  const double t = block_sum<256>(v, s_wave);
  if (threadIdx.x == 0) part[piece0 + blockIdx.x] = t;
}

// c = coef[0] coef[1]: 1 and c, or, where c is near or under fp32's smallest normal value, a power of two
// and a factor that are both well inside the range (huge gradients clipped to a tiny norm: c as one fp32
// value would keep a few of its 24 bits, or none).
__global__ __launch_bounds__(1024) void k_norm(const double* __restrict__ part, int64_t pieces, float max_norm,
                                               float* __restrict__ norm, float* __restrict__ coef) {
  __shared__ double s_wave[16];
  double v = 0.0;
  for (int64_t i = threadIdx.x; i < pieces; i += 1024) v += part[i];
  const double t = block_sum<1024>(v, s_wave);
  if (threadIdx.x == 0) {
    const double nrm = sqrt(t);
    const double c = (double)max_norm / (nrm + 1e-6);
    const double used = max_norm == INFINITY || c > 1.0 ? 1.0 : c;           // NaN stays, but for the norm alone
    const double scale = used > 0.0 && used < 0x1p-100 ? ldexp(1.0, ilogb(used) / 2) : 1.0;
    *norm = (float)nrm;
    coef[0] = (float)scale;
    coef[1] = (float)(used / scale);
  }
}

template <typename T>
__device__ __forceinline__ void scaled(const T* p, T* o, int n, bool vec, float scale, float c) {
  Chunk<T> q;
  q.load(p, n, vec);
#pragma unroll
  for (int j = 0; j < Chunk<T>::kLoads; ++j) {
    const int at = j * 256 + threadIdx.x;
    if (at * Chunk<T>::kEach >= q.whole) break;
    uint32_t e[4] = {q.w[j].x, q.w[j].y, q.w[j].z, q.w[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) e[i] = __float_as_uint(c * (scale * __uint_as_float(e[i])));
      else e[i] = pack_bf16(c * (scale * bf16_lo(e[i])), c * (scale * bf16_hi(e[i])));
    }
    reinterpret_cast<uint4*>(o)[at] = make_uint4(e[0], e[1], e[2], e[3]);
  }
#pragma unroll 4
  for (int i = q.whole + threadIdx.x; i < n; i += 256) store_out(o, i, c * (scale * value(p[i])));
}

__global__ __launch_bounds__(256) void k_scale(const ClipItem* __restrict__ table, int count, int64_t pieces,
                                               int64_t piece0, const float* __restrict__ coef) {
  const float scale = coef[0], c = coef[1];
  const Piece q = find_piece(table, count, pieces, piece0 + blockIdx.x);
  if (scale == 1.f && c == 1.f && q.out == q.g) return;
  if (q.bf16) scaled(static_cast<const uint16_t*>(q.g) + q.i0, static_cast<uint16_t*>(q.out) + q.i0, q.n, q.vec, scale, c);
  else scaled(static_cast<const float*>(q.g) + q.i0, static_cast<float*>(q.out) + q.i0, q.n, q.vec, scale, c);
}

int64_t clip_pieces(int64_t numel) { return (numel + kPiece - 1) / kPiece; }
int clip_tail(int64_t numel) { return (int)(numel - (clip_pieces(numel) - 1) * kPiece); }

hipError_t launch_clip_table(const ClipGroup& grp, ClipItem* table, hipStream_t s) {
  hipLaunchKernelGGL(k_table, dim3(1), dim3(64), 0, s, grp, table);
  return hipGetLastError();
}

// 2^23 pieces to a launch (2^32 work-items are too many for one).
constexpr int64_t kLaunchPieces = int64_t(1) << 23;

hipError_t launch_clip_square(const ClipItem* table, int count, int64_t pieces, double* part, hipStream_t s) {
  for (int64_t p = 0; p < pieces; p += kLaunchPieces)
    hipLaunchKernelGGL(k_square, dim3((unsigned)std::min(kLaunchPieces, pieces - p)), dim3(256), 0, s, table, count, pieces,
                       p, part);
  return hipGetLastError();
}

hipError_t launch_clip_norm(const double* part, int64_t pieces, float max_norm, float* norm, float* coef, hipStream_t s) {
  hipLaunchKernelGGL(k_norm, dim3(1), dim3(1024), 0, s, part, pieces, max_norm, norm, coef);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipItem* table, int count, int64_t pieces, const float* coef, hipStream_t s) {
  for (int64_t p = 0; p < pieces; p += kLaunchPieces)
    hipLaunchKernelGGL(k_scale, dim3((unsigned)std::min(kLaunchPieces, pieces - p)), dim3(256), 0, s, table, count, pieces,
                       p, coef);
  return hipGetLastError();
}

}  // namespace f2i
