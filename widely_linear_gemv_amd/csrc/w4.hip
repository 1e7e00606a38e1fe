// Decode products with layers kept at four bits: codes c in 0..15, a scale s and a zero point z for each
// row and group of G columns,
//
//     W_ij = s_i,j/G (c_ij - z_i,j/G)        y_bi = sum_j W_ij x_bj
//
// On the bf16 matrix cores: a code becomes the bf16 value 1 + c / 16 by a shift and one and-or for two of
// them (its bits are the top of the significand), so within a group
//     sum_j (c_j - z) x_j = 16 (sum_j (1 + c_j / 16) x_j - (1 + z / 16) sum_j x_j)
// with exact products, fp32 sums, and sum_j x_j made once per workgroup.  (The value 128 + c takes the same
// instructions but leaves five bits less of the sums.)  fp32 x enters as three bf16 parts that hold it.
//
// Packed form: tiles of 16 rows, one after another; a tile's codes are 1 KB blocks of 128 columns, and in a
// block lane l = 16 g + r of a wave owns the 16 bytes of row r: word s holds columns 32 s + 8 g + e, e < 8, of
// the block, e even in nibble e / 2 and e odd in nibble 4 + e / 2, as the matrix instruction's operand takes
// them.  Behind all codes, for each tile and group: the 16 rows' scales, then their 16 zero points (a byte each).
#include <algorithm>

#include "tiles.hpp"

namespace f2i {

namespace {

constexpr int kChunk = 128;              // columns of a block of codes
constexpr int kWaves = 8;
constexpr int kLdsX = 56 * 1024;         // bytes of x that a workgroup holds at once

__host__ __device__ __forceinline__ int64_t w4_tiles(int64_t rows) { return (rows + 15) / 16; }
__host__ __device__ __forceinline__ int64_t w4_chunks(int64_t cols) { return (cols + kChunk - 1) / kChunk; }
__host__ __device__ __forceinline__ int w4_group_bytes(int scale_bytes) { return 16 * scale_bytes + 16; }

// One word of codes a thread.
__global__ __launch_bounds__(256) void k_w4_codes(const uint8_t* __restrict__ codes, int64_t rows, int64_t cols,
                                                  int64_t chunks, int64_t words, uint32_t* __restrict__ out) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= words) return;
  const int s = at & 3, lane = (at >> 2) & 63;
  const int64_t block = at >> 8, tile = block / chunks, chunk = block - tile * chunks;
  const int64_t i = tile * 16 + (lane & 15), j = chunk * kChunk + 32 * s + 8 * (lane >> 4);
  uint32_t w = 0;
  if (i < rows) {
    const uint8_t* __restrict__ p = codes + i * cols + j;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e < cols) w |= (uint32_t)(p[e] & 15) << (4 * ((e >> 1) + 4 * (e & 1)));
  }
  out[at] = w;
}

// One row of one tile and group a thread.
template <typename ST>
__global__ __launch_bounds__(256) void k_w4_scales(const ST* __restrict__ scales, const uint8_t* __restrict__ zeros,
                                                   int64_t rows, int64_t groups, int64_t count,
                                                   uint8_t* __restrict__ out) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= count) return;
  const int r = at & 15;
  const int64_t block = at >> 4, tile = block / groups, group = block - tile * groups;
  const int64_t i = tile * 16 + r;
  uint8_t* __restrict__ to = out + block * w4_group_bytes(sizeof(ST));
  reinterpret_cast<ST*>(to)[r] = i < rows ? scales[i * groups + group] : ST(0);
  to[16 * sizeof(ST) + r] = i < rows && zeros ? zeros[i * groups + group] : 8;
}

// Four rows' scales times 16, and 1 + z / 16.
template <typename ST>
struct RowScales {
  v4f s, z;
  __device__ __forceinline__ void load(const uint8_t* group, int g) {
    if constexpr (sizeof(ST) == 2) {
      const uint2 w = *reinterpret_cast<const uint2*>(group + 8 * g);
      s = v4f{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
    } else {
      s = *reinterpret_cast<const v4f*>(group + 16 * g);
    }
    const uint32_t b = *reinterpret_cast<const uint32_t*>(group + 16 * sizeof(ST) + 4 * g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] *= 16.f;
      z[e] = fmaf((float)((b >> (8 * e)) & 255), 0.0625f, 1.f);
    }
  }
};

// Eight codes as an operand.
__device__ __forceinline__ v4u codes_bf16(uint32_t w) {
  constexpr uint32_t kMask = 0x00780078u, kOne = 0x3F803F80u;
  return v4u{((w << 3) & kMask) | kOne, ((w >> 1) & kMask) | kOne, ((w >> 5) & kMask) | kOne, ((w >> 9) & kMask) | kOne};
}

__device__ __forceinline__ float wide(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float wide(float v) { return v; }

struct W4Kernel {
  const uint8_t* packed;
  const void* x;
  void* y;
  int64_t rows, cols, chunks, groups;
  int B, seg;            // seg: columns of x held at once, a multiple of 128
};

// A workgroup per tile; its waves take the blocks of codes in turn, and their sums meet in LDS in wave
// order.  x lies in LDS, `seg` columns at a time, each batch entry's row 16 bytes longer than its data (the
// sixteen entries of an operand read then cover the banks evenly).
template <int G, typename XT, typename ST, typename YT>
__global__ __launch_bounds__(64 * kWaves) void k_w4(W4Kernel t) {
  constexpr int kParts = sizeof(XT) == 2 ? 1 : 3;
  extern __shared__ __align__(16) uint8_t s_mem[];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int64_t tile = blockIdx.x;
  const int pitch = t.seg * 2 + 16;                                    // bytes
  const int plane = pitch * t.B;
  float* s_sum = reinterpret_cast<float*>(s_mem + kParts * plane);     // [B][seg / G]
  const int sums = t.seg / G;
  const uint8_t* scales = t.packed + w4_tiles(t.rows) * t.chunks * 1024 + tile * t.groups * w4_group_bytes(sizeof(ST));
  const v4u* codes = reinterpret_cast<const v4u*>(t.packed + tile * t.chunks * 1024) + lane;
  const int entry = min(c, t.B - 1);                                   // columns past the batch are not stored
  v4f y = v4f{0.f, 0.f, 0.f, 0.f};
  for (int64_t k0 = 0; k0 < t.cols; k0 += t.seg) {
    if (k0 > 0) __syncthreads();
    // x and its group sums
    for (int u = tid; u < t.B * t.seg / 8; u += 64 * kWaves) {
      const int b = u / (t.seg / 8), k = (u - b * (t.seg / 8)) * 8;
      const XT* __restrict__ from = static_cast<const XT*>(t.x) + b * t.cols + k0 + k;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = k0 + k + e < t.cols ? wide(from[e]) : 0.f;
      float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        v4u w;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float a = f[2 * h], d = f[2 * h + 1];
          if (kParts > 1 && p == 0) {                                   // a value past the largest bf16
            constexpr float kMost = 0x1.FEp127f;
            a = __builtin_amdgcn_fmed3f(a, -kMost, kMost);
            d = __builtin_amdgcn_fmed3f(d, -kMost, kMost);
          }
          w[h] = pack_bf16(a, d);
          f[2 * h] -= bf16_lo(w[h]);
          f[2 * h + 1] -= bf16_hi(w[h]);
        }
        *reinterpret_cast<v4u*>(s_mem + p * plane + b * pitch + k * 2) = w;
      }
      sum = group_sum<G / 8>(sum);
      if (k % G == 0) s_sum[b * sums + k / G] = sum;
    }
    __syncthreads();
    const int64_t c0 = k0 / kChunk, c1 = min(c0 + t.seg / kChunk, t.chunks);
    for (int64_t ch = c0 + ((wave - c0) & (kWaves - 1)); ch < c1; ch += kWaves) {   // wave ch % 8, whatever seg is
      const v4u w = codes[ch * 64];
      const uint8_t* xs = s_mem + entry * pitch + (int)(ch - c0) * kChunk * 2 + 16 * g;
      const float* sum = s_sum + entry * sums + (int)(ch - c0) * (kChunk / G);
#pragma unroll
      for (int q = 0; q < kChunk / G; ++q) {
        RowScales<ST> rs;
        rs.load(scales + min(ch * (kChunk / G) + q, t.groups - 1) * w4_group_bytes(sizeof(ST)), g);
        v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = q * (G / 32); s < (q + 1) * (G / 32); ++s) {
          const v4u a = codes_bf16(w[s]);
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p)
            acc = Mma<uint16_t>::run(a, *reinterpret_cast<const v4u*>(xs + p * plane + s * 64), acc);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = fmaf(rs.s[e], fmaf(-rs.z[e], sum[q], acc[e]), y[e]);
      }
    }
  }
  __syncthreads();
  // [wave][entry][row]
  float* s_y = reinterpret_cast<float*>(s_mem);
  if (c < t.B) *reinterpret_cast<v4f*>(s_y + (wave * t.B + c) * 16 + 4 * g) = y;
  __syncthreads();
  if (tid < t.B * 16) {
    float v = s_y[tid];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += s_y[w * t.B * 16 + tid];
    const int64_t i = tile * 16 + (tid & 15);
    if (i < t.rows) store_out(static_cast<YT*>(t.y), (tid >> 4) * t.rows + i, v);
  }
}

template <int G, typename XT, typename ST, typename YT>
hipError_t w4_gemv_t(const W4Args& a, hipStream_t s) {
  constexpr int kParts = sizeof(XT) == 2 ? 1 : 3;
  W4Kernel t{a.packed, a.x, a.y, a.rows, a.cols, w4_chunks(a.cols), (a.cols + G - 1) / G, a.B, 0};
  const int64_t fit = kLdsX / a.B / (2 * kParts) / kChunk * kChunk;
  t.seg = (int)std::min<int64_t>(fit, t.chunks * kChunk);
  const size_t lds = std::max<size_t>((size_t)a.B * ((t.seg * 2 + 16) * kParts + t.seg / G * 4), (size_t)kWaves * a.B * 64);
  hipLaunchKernelGGL((k_w4<G, XT, ST, YT>), dim3((unsigned)w4_tiles(a.rows)), dim3(64 * kWaves), lds, s, t);
  return hipGetLastError();
}

template <int G, typename XT, typename ST>
hipError_t w4_gemv_y(const W4Args& a, hipStream_t s) {
  return a.y_bf16 ? w4_gemv_t<G, XT, ST, uint16_t>(a, s) : w4_gemv_t<G, XT, ST, float>(a, s);
}
template <int G>
hipError_t w4_gemv_g(const W4Args& a, hipStream_t s) {
  if (a.x_bf16) return a.scales_bf16 ? w4_gemv_y<G, uint16_t, uint16_t>(a, s) : w4_gemv_y<G, uint16_t, float>(a, s);
  return a.scales_bf16 ? w4_gemv_y<G, float, uint16_t>(a, s) : w4_gemv_y<G, float, float>(a, s);
}

}  // namespace

size_t w4_bytes(int64_t rows, int64_t cols, int group, int scales_bf16) {
  return (size_t)w4_tiles(rows) *
         (w4_chunks(cols) * 1024 + (cols + group - 1) / group * w4_group_bytes(scales_bf16 ? 2 : 4));
}

hipError_t launch_w4_pack(const uint8_t* codes, const void* scales, int scales_bf16, const uint8_t* zeros, int64_t rows,
                          int64_t cols, int group, uint8_t* packed, hipStream_t s) {
  const int64_t chunks = w4_chunks(cols), words = w4_tiles(rows) * chunks * 256;
  const int64_t groups = (cols + group - 1) / group, count = w4_tiles(rows) * groups * 16;
  hipLaunchKernelGGL(k_w4_codes, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s, codes, rows, cols, chunks, words,
                     reinterpret_cast<uint32_t*>(packed));
  const dim3 grid((unsigned)((count + 255) / 256));
  if (scales_bf16)
    hipLaunchKernelGGL((k_w4_scales<uint16_t>), grid, dim3(256), 0, s, static_cast<const uint16_t*>(scales), zeros, rows,
                       groups, count, packed + words * 4);
  else
    hipLaunchKernelGGL((k_w4_scales<float>), grid, dim3(256), 0, s, static_cast<const float*>(scales), zeros, rows, groups,
                       count, packed + words * 4);
  return hipGetLastError();
}

hipError_t launch_w4_gemv(const W4Args& a, hipStream_t s) {
  switch (a.group) {
    case 32: return w4_gemv_g<32>(a, s);
    case 64: return w4_gemv_g<64>(a, s);
    default: return w4_gemv_g<128>(a, s);
  }
}

}  // namespace f2i
