// Global gradient norm over many tensors, and clipping:
//     norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c g.
//
// Squares and sums are fp64 (the vector ALUs do far more fp64 adds per second than HBM delivers
// values), so no gradient is large or small enough to over- or underflow the sum.  Three passes:
// k_square writes one partial sum per 8192-element piece, k_norm joins them in a fixed order (the
// result never depends on scheduling) into the norm and c, k_scale multiplies.  The norm must be
// known before the first write, so the gradients are read twice; the second time they come from
// the Infinity Cache as far as they fit.  In place with c = 1 nothing is written.
#include "common.hpp"

namespace f2i {

namespace {

constexpr int kPiece = 8192;       // elements per workgroup

// Tensor of workgroup `block`: the last one whose first piece is at or before it.
__device__ __forceinline__ int find_tensor(const ClipGroup& g, int block) {
  int lo = 0, hi = g.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.items[mid].first_piece <= block) lo = mid; else hi = mid - 1;
  }
  return lo;
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

__global__ __launch_bounds__(256) void k_square(ClipGroup grp, double* __restrict__ part) {
  __shared__ double s_wave[4];
  const int k = find_tensor(grp, blockIdx.x);
  const ClipItem& it = grp.items[k];
  const int64_t i0 = (int64_t)(blockIdx.x - it.first_piece) * kPiece;
  const int n = (int)min((int64_t)kPiece, it.numel - i0);
  double v = 0.0;
  if (it.bf16) {
    const uint16_t* __restrict__ p = static_cast<const uint16_t*>(it.g) + i0;
    int i = threadIdx.x;
    if (it.vec) {
      for (i = threadIdx.x * 8; i + 8 <= n; i += 256 * 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(p + i);
        v += sq(bf16_lo(w.x)) + sq(bf16_hi(w.x)) + sq(bf16_lo(w.y)) + sq(bf16_hi(w.y));
        v += sq(bf16_lo(w.z)) + sq(bf16_hi(w.z)) + sq(bf16_lo(w.w)) + sq(bf16_hi(w.w));
      }
      i = (n & ~7) + threadIdx.x;
    }
    for (; i < n; i += 256) v += sq(bf16_lo(p[i]));
  } else {
    const float* __restrict__ p = static_cast<const float*>(it.g) + i0;
    int i = threadIdx.x;
    if (it.vec) {
      for (i = threadIdx.x * 4; i + 4 <= n; i += 256 * 4) {
        const float4 w = *reinterpret_cast<const float4*>(p + i);
        v += (sq(w.x) + sq(w.y)) + (sq(w.z) + sq(w.w));
      }
      i = (n & ~3) + threadIdx.x;
    }
    for (; i < n; i += 256) v += sq(p[i]);
  }
  const double t = block_sum<256>(v, s_wave);
  if (threadIdx.x == 0) part[grp.piece0 + blockIdx.x] = t;
}

// coef[0] = c (fp32).
__global__ __launch_bounds__(1024) void k_norm(const double* __restrict__ part, int64_t pieces, float max_norm,
                                               float* __restrict__ norm, float* __restrict__ coef) {
  __shared__ double s_wave[16];
  double v = 0.0;
  for (int64_t i = threadIdx.x; i < pieces; i += 1024) v += part[i];
  const double t = block_sum<1024>(v, s_wave);
  if (threadIdx.x == 0) {
    const double nrm = sqrt(t);
    const double c = (double)max_norm / (nrm + 1e-6);
    *norm = (float)nrm;
    *coef = (float)(c > 1.0 ? 1.0 : c);        // NaN stays
  }
}

__global__ __launch_bounds__(256) void k_scale(ClipGroup grp, const float* __restrict__ coef) {
  const int k = find_tensor(grp, blockIdx.x);
  const ClipItem& it = grp.items[k];
  const float c = *coef;
  if (c == 1.f && it.out == it.g) return;
  const int64_t i0 = (int64_t)(blockIdx.x - it.first_piece) * kPiece;
  const int n = (int)min((int64_t)kPiece, it.numel - i0);
  if (it.bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(it.g) + i0;
    uint16_t* o = static_cast<uint16_t*>(it.out) + i0;
    int i = threadIdx.x;
    if (it.vec) {
      for (i = threadIdx.x * 8; i + 8 <= n; i += 256 * 8) {
        uint4 w = *reinterpret_cast<const uint4*>(p + i);
        uint32_t* e = &w.x;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          e[j] = (uint32_t)f32_to_bf16_rne(c * bf16_lo(e[j])) | ((uint32_t)f32_to_bf16_rne(c * bf16_hi(e[j])) << 16);
        *reinterpret_cast<uint4*>(o + i) = w;
      }
      i = (n & ~7) + threadIdx.x;
    }
    for (; i < n; i += 256) o[i] = f32_to_bf16_rne(c * bf16_lo(p[i]));
  } else {
    const float* p = static_cast<const float*>(it.g) + i0;
    float* o = static_cast<float*>(it.out) + i0;
    int i = threadIdx.x;
    if (it.vec) {
      for (i = threadIdx.x * 4; i + 4 <= n; i += 256 * 4) {
        const float4 w = *reinterpret_cast<const float4*>(p + i);
        *reinterpret_cast<float4*>(o + i) = make_float4(c * w.x, c * w.y, c * w.z, c * w.w);
      }
      i = (n & ~3) + threadIdx.x;
    }
    for (; i < n; i += 256) o[i] = c * p[i];
  }
}

int64_t clip_pieces(int64_t numel) { return (numel + kPiece - 1) / kPiece; }

hipError_t launch_clip_square(const ClipGroup& grp, int pieces, double* part, hipStream_t s) {
  hipLaunchKernelGGL(k_square, dim3(pieces), dim3(256), 0, s, grp, part);
  return hipGetLastError();
}

hipError_t launch_clip_norm(const double* part, int64_t pieces, float max_norm, float* norm, float* coef, hipStream_t s) {
  hipLaunchKernelGGL(k_norm, dim3(1), dim3(1024), 0, s, part, pieces, max_norm, norm, coef);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipGroup& grp, int pieces, const float* coef, hipStream_t s) {
  hipLaunchKernelGGL(k_scale, dim3(pieces), dim3(256), 0, s, grp, coef);
  return hipGetLastError();
}

}  // namespace f2i
