// Decode products with layers kept at four bits: codes c in 0..15, a scale s and a zero point z for each
// row and group of G columns,
//
//     W_ij = s_i,j/G (c_ij - z_i,j/G)        y_bi = sum_j W_ij x_bj
//
// On the bf16 matrix cores, with exact products and fp32 sums.  bf16 x: a code becomes the bf16 value 1 + c / 16 by
// a shift and one and-or for two of them (its bits are the top of the significand), so within a group
//     sum_j (c_j - z) x_j = 16 (sum_j (1 + c_j / 16) x_j - (1 + z / 16) sum_j x_j)
// with sum_j x_j made once for a workgroup's tiles.  (The value 128 + c takes the same instructions but leaves five
// bits less of the sums.)  The two sums are larger than their difference; outputs are 1.0e-7 to 2.3e-7 of their norm
// off, for x of mean 3 0.5e-7 to 1.0e-7, less than an fp32 product with the matrix written out (2.2e-7 to 9e-7).
// fp32 x enters as three bf16 parts that hold it, so that three times as many roundings count: there a code becomes
// c - z itself, exact in bf16 for every byte z (4.75 instructions for two codes instead of 1.75).  A weight that is
// 0 then adds 0, and outputs are 1.2e-7 off instead of 3.5e-7 to 1.3e-6, for x of mean 3 1.0e-7 instead of 5e-7 to
// 1.9e-6 (the matrix written out 3e-7 to 11e-7).  It costs 0.1-1.7 us: 4096 x 4096, one entry 7.1 -> 7.2 us; 11008 x
// 4096, 16 entries 14.9 -> 16.2, one entry 10.8 -> 12.5.  (With bf16 x the same would cost 32000 x 4096, one entry,
// 14.4 -> 17.2 us.)
//
// Packed form: tiles of 16 rows, one after another, each in blocks of 128 columns.  A block is 1 KB of codes,
// then its scales, then its zero points.  In the codes lane l = 16 g + r of a wave owns the 16 bytes of row r:
// word s holds columns 32 s + 8 g + e, e < 8, of the block, e even in nibble e / 2 and e odd in nibble
// 4 + e / 2, the whole word rotated left by 3 bits: nibbles n and n + 4 are then two neighbouring values of the
// matrix instruction's operand after a rotation by 4 n.  Scales and zero points (a byte each) are ordered
// [row][group of the block].
#include <algorithm>

#include "tiles.hpp"

namespace f2i {

namespace {

constexpr int kChunk = 128;              // columns of a block

__host__ __device__ __forceinline__ int64_t w4_tiles(int64_t rows) { return (rows + 15) / 16; }
__host__ __device__ __forceinline__ int64_t w4_chunks(int64_t cols) { return (cols + kChunk - 1) / kChunk; }
__host__ __device__ __forceinline__ constexpr int w4_block_bytes(int group, int scale_bytes) {
  return 1024 + kChunk / group * 16 * (scale_bytes + 1);
}

// One word of codes a thread.  32000 x 4096 with its scales in 44 us (133 MB read, 68 written: 4.6 TB/s).
__global__ __launch_bounds__(256) void k_w4_codes(const uint8_t* __restrict__ codes, int64_t rows, int64_t cols,
                                                  int64_t chunks, int64_t words, int block_bytes,
                                                  uint8_t* __restrict__ out) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= words) return;
  const int s = at & 3, lane = (at >> 2) & 63;
  const int64_t block = at >> 8, tile = block / chunks, chunk = block - tile * chunks;
  const int64_t i = tile * 16 + (lane & 15), j = chunk * kChunk + 32 * s + 8 * (lane >> 4);
  uint32_t w = 0;
  if (i < rows) {
    const uint8_t* __restrict__ p = codes + i * cols + j;
    uint32_t c[2] = {0, 0};                      // columns j .. j + 3 and j + 4 .. j + 7, a byte each
    if (j + 8 <= cols) {
      __builtin_memcpy(c, p, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < cols) c[e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= (c[e / 4] >> (8 * (e % 4)) & 15) << (4 * ((e >> 1) + 4 * (e & 1)));
  }
  *reinterpret_cast<uint32_t*>(out + block * block_bytes + (at & 255) * 4) = w << 3 | w >> 29;
}

// One row of one block and group a thread.
template <typename ST>
__global__ __launch_bounds__(256) void k_w4_scales(const ST* __restrict__ scales, const uint8_t* __restrict__ zeros,
                                                   int64_t rows, int64_t groups, int64_t chunks, int each, int64_t count,
                                                   int block_bytes, uint8_t* __restrict__ out) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;      // [block][row][group of the block]
  if (at >= count) return;
  const int64_t block = at / (16 * each), tile = block / chunks, chunk = block - tile * chunks;
  const int in = (int)(at - block * 16 * each);
  const int64_t i = tile * 16 + in / each, group = chunk * each + in % each;
  const bool have = i < rows && group < groups;
  uint8_t* __restrict__ to = out + block * block_bytes + 1024;
  reinterpret_cast<ST*>(to)[in] = have ? scales[i * groups + group] : ST(0);
  to[16 * each * sizeof(ST) + in] = have && zeros ? zeros[i * groups + group] : 8;
}

// Eight codes as an operand.  (The masks are kept in registers: as literals they cost an instruction more.)
template <bool EXACT>
struct Codes {
  uint32_t bits = 0x00780078u, one = EXACT ? 0x64006400u : 0x3F803F80u;
  __device__ __forceinline__ Codes() { asm volatile("" : "+s"(bits), "+v"(one)); }
  __device__ __forceinline__ uint32_t two(uint32_t w, int n) const {           // nibbles n and n + 4
    return ((n < 3 ? w >> (4 * n) : __builtin_amdgcn_alignbit(w, w, 12)) & bits) | one;
  }
  // 1 + c / 16
  __device__ __forceinline__ v4u plain(uint32_t w) const { return v4u{two(w, 0), two(w, 1), two(w, 2), two(w, 3)}; }
  // c - z from the fp16 value 1024 + 8 c
  __device__ __forceinline__ v4u minus(uint32_t w, float z) const {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    const float off = -128.f - z;
    v4u out;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const v2h h = __builtin_bit_cast(v2h, two(w, n));
      out[n] = pack_bf16(fmaf((float)h[0], 0.125f, off), fmaf((float)h[1], 0.125f, off));
    }
    return out;
  }
};

// A load of 16 bytes at any element's alignment.
struct __attribute__((packed, aligned(2))) Any16 {
  v4u v;
};

// One wave's block of x: 128 columns of ROWS batch entries, read in whole cache lines (a wave instruction
// reads 256 bytes of four rows of bf16, 512 of two of fp32) and turned in LDS into the matrix instruction's operand.
// A row there is 16 bytes longer than its data, so that the sixteen rows of an operand read lie in distinct
// banks.  fp32 is cut into three bf16 parts that hold it on the way, the largest first.
template <typename XT, int ROWS>
struct XBlock {
  static constexpr int kParts = sizeof(XT) == 2 ? 1 : 3;
  static constexpr int kPitch = 2 * kChunk + 16, kPlane = ROWS * kPitch;
  static constexpr int kLanes = kChunk * sizeof(XT) / 16;            // of a row
  static constexpr int kLoads = ROWS * kLanes / kWave;
  static constexpr int kEach = 16 / sizeof(XT);                      // values of a lane's load
  v4u raw[kLoads];
  // offset in elements of a lane's piece in load i
  __device__ static __forceinline__ uint32_t offset(int i, int lane, int B, int64_t cols) {
    return (uint32_t)(min(i * (kWave / kLanes) + lane / kLanes, B - 1) * cols) + lane % kLanes * kEach;
  }
  __device__ __forceinline__ void load(const XT* x, const uint32_t (&off)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw[i] = reinterpret_cast<const Any16*>(x + off[i])->v;
  }
  __device__ __forceinline__ void load_end(const XT* x, const uint32_t (&off)[kLoads], int have) {   // the first `have` columns
    const int mine = have - (int)(threadIdx.x & (kLanes - 1)) * kEach;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(XT) == 4) {
          raw[i][e] = e < mine ? __float_as_uint(x[off[i] + e]) : 0;
        } else {
          const uint32_t lo = 2 * e < mine ? x[off[i] + 2 * e] : 0, hi = 2 * e + 1 < mine ? x[off[i] + 2 * e + 1] : 0;
          raw[i][e] = lo | hi << 16;
        }
      }
  }
  __device__ __forceinline__ void store(uint8_t* lds, int lane) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint8_t* to = lds + (i * (kWave / kLanes) + lane / kLanes) * kPitch + lane % kLanes * kEach * 2;
      if constexpr (sizeof(XT) == 2) {
        *reinterpret_cast<v4u*>(to) = raw[i];
      } else {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(raw[i][e]);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          constexpr float kMost = 0x1.FEp127f;                       // a value past the largest bf16
          v2u w;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = f[2 * h], b = f[2 * h + 1];
            w[h] = p == 0 ? pack_bf16(__builtin_amdgcn_fmed3f(a, -kMost, kMost), __builtin_amdgcn_fmed3f(b, -kMost, kMost))
                          : pack_bf16(a, b);
            f[2 * h] -= bf16_lo(w[h]);
            f[2 * h + 1] -= bf16_hi(w[h]);
          }
          *reinterpret_cast<v2u*>(to + p * kPlane) = w;
        }
      }
    }
  }
};

// Scales and zero points of a row in a block: N groups.
template <int N, typename ST>
struct RowScales {
  struct __attribute__((packed, aligned(N * sizeof(ST)))) S { ST v[N]; } s;
  struct __attribute__((packed, aligned(N))) Z { uint8_t v[N]; } z;
  __device__ __forceinline__ void load(const uint8_t* block, int row) {
    s = *reinterpret_cast<const S*>(block + 1024 + row * N * sizeof(ST));
    z = *reinterpret_cast<const Z*>(block + 1024 + 16 * N * sizeof(ST) + row * N);
  }
  __device__ __forceinline__ float scale(int q) const {
    if constexpr (sizeof(ST) == 4) return s.v[q];
    else return __uint_as_float((uint32_t)s.v[q] << 16);
  }
  __device__ __forceinline__ float zero(int q) const { return (float)z.v[q]; }
};

struct W4Kernel {
  const uint8_t* packed;
  const void* x;
  void* y;
  int64_t rows, cols, chunks, tiles;
  int B, y_bf16;
};

// Bound by HBM for few entries (32000 x 4096, 68 MB: 13.4-15.1 us, 4.5-5.1 TB/s; all loads without products or x at
// 65536 columns 5.5 TB/s), by the launch for small layers (4096 x 4096, 8.7 MB: 4.2 us of which 2.6 are left
// without any data to speak of), and for sixteen entries by the chain of a wave's blocks: it waits for one, turns x
// in LDS, multiplies, and loads the next.  A round of 2048 columns of 4096 rows takes 1.0 us for one entry, 1.6-1.8
// for sixteen (4096 x 11008: 11.5 us for 26 MB of codes and 90 MB of x, 14-21 bytes a clock and CU, which the L2 has
// more of); with fp32 x one of 1024 columns 1.2 and 1.75.
// A workgroup of NW waves for RT tiles of 16 rows and all of the batch: the waves take the blocks of columns in
// turn and their sums meet in LDS in wave order.  Batch entries are the rows of the product, so that a lane
// holds one weight row's sums for four entries and needs that row's scales alone.
template <int G, typename XT, typename ST, int NW, int RT, int ROWS, int NB>
__global__ __launch_bounds__(64 * NW) void k_w4(W4Kernel t) {
  constexpr int kBlock = w4_block_bytes(G, sizeof(ST)), kGroups = kChunk / G;
  using X = XBlock<XT, ROWS>;
  constexpr int kMine = X::kParts * X::kPlane;                       // a wave's bytes of LDS
  constexpr int kSums = RT * ROWS * 64;                              // and of its sums, which take over
  __shared__ __align__(16) uint8_t s_mem[NW * (kMine > kSums ? kMine : kSums)];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int64_t tile0 = (int64_t)blockIdx.x * RT;
  const XT* __restrict__ x = static_cast<const XT*>(t.x);
  uint32_t off[X::kLoads];
#pragma unroll
  for (int i = 0; i < X::kLoads; ++i) off[i] = X::offset(i, lane, t.B, t.cols);
  uint8_t* mine_x = s_mem + wave * kMine;
  const uint8_t* operand = mine_x + min(c, t.B - 1) * X::kPitch + 16 * g;      // entries past the batch are not stored
  const uint8_t* base[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) base[r] = t.packed + min(tile0 + r, t.tiles - 1) * t.chunks * kBlock;
  struct Block {
    v4u w[RT];
    RowScales<kGroups, ST> s[RT];
    X x;
  };
  auto load_codes = [&](Block& b, int ch) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint8_t* at = base[r] + (int64_t)ch * kBlock;
      b.w[r] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(at + lane * 16));
      b.s[r].load(at, c);
    }
  };
  float y[RT][NB];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int e = 0; e < NB; ++e) y[r][e] = 0.f;
  constexpr bool kExact = sizeof(XT) == 4;
  const Codes<kExact> codes;
  auto multiply = [&](const Block& b) {
    const v4u one = v4u{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    asm volatile("" ::: "memory");                       // a wave's reads and writes of LDS stay in their order
    b.x.store(mine_x, lane);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      v4f acc[RT], sum = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = q * (G / 32); s < (q + 1) * (G / 32); ++s) {
        v4u w[RT];
        if constexpr (kExact)
#pragma unroll
          for (int r = 0; r < RT; ++r) w[r] = codes.minus(b.w[r][s], b.s[r].zero(q));
#pragma unroll
        for (int p = X::kParts - 1; p >= 0; --p) {
          const v4u xp = *reinterpret_cast<const v4u*>(operand + p * X::kPlane + 64 * s);
          if constexpr (!kExact) sum = Mma<uint16_t>::run(xp, one, sum);
#pragma unroll
          for (int r = 0; r < RT; ++r)
            acc[r] = Mma<uint16_t>::run(xp, kExact ? w[r] : codes.plain(b.w[r][s]), acc[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float z = fmaf(b.s[r].zero(q), -0.0625f, -1.f), scale = b.s[r].scale(q);
#pragma unroll
        for (int e = 0; e < NB; ++e)
          y[r][e] = kExact ? fmaf(scale, acc[r][e], y[r][e]) : fmaf(16.f * scale, fmaf(z, sum[e], acc[r][e]), y[r][e]);
      }
    }
  };
  const int whole = (int)(t.cols / kChunk);
  Block b;
  for (int ch = wave; ch < whole; ch += NW) {
    load_codes(b, ch);
    b.x.load(x + ch * kChunk, off);
    multiply(b);
  }
  if (whole < t.chunks && whole % NW == wave) {                          // the last block, of fewer columns
    load_codes(b, whole);
    b.x.load_end(x + whole * kChunk, off, (int)t.cols - whole * kChunk);
    multiply(b);
  }
  __syncthreads();
  float* s_y = reinterpret_cast<float*>(s_mem);                      // [wave][tile][entry][row]
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int e = 0; e < NB; ++e)
      if (4 * g + e < t.B) s_y[((wave * RT + r) * ROWS + 4 * g + e) * 16 + c] = y[r][e];
  __syncthreads();
  for (int k = tid; k < RT * t.B * 16; k += NW * kWave) {
    const int r = k / (t.B * 16), at = k - r * t.B * 16;
    float v = s_y[r * ROWS * 16 + at];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += s_y[(w * RT + r) * ROWS * 16 + at];
    const int64_t i = (tile0 + r) * 16 + (at & 15), to = (at >> 4) * t.rows + i;
    if (i >= t.rows) continue;
    if (t.y_bf16) store_out(static_cast<uint16_t*>(t.y), to, v);
    else store_out(static_cast<float*>(t.y), to, v);
  }
}

template <int G, typename XT, typename ST, int NW, int RT, int ROWS, int NB>
void w4_run(const W4Kernel& t, hipStream_t s) {
  hipLaunchKernelGGL((k_w4<G, XT, ST, NW, RT, ROWS, NB>), dim3((unsigned)((t.tiles + RT - 1) / RT)), dim3(64 * NW), 0, s, t);
}

// Waves to a tile (NW) and tiles to a workgroup (RT).  One block of codes in flight a wave, and as many waves
// on a CU as its registers hold, beat fewer waves with two to eight blocks in flight by 5-30 % where there are
// tiles for them (32000 x 4096, one entry: 14.2-15.1 us, with two blocks 17.6, four 19.7; not measured up to a tile a
// CU, where the grid and not the registers bounds the waves).  Up to a tile a CU sixteen waves share a tile (4096
// x 4096, one entry: 16 waves 4.3 us, 8 waves 5.2; 4096 x 11008, 16 entries 11.6 and 11.8), beyond that eight
// (6144 x 4096: 8 waves 5.8, 16 waves 6.7; 32000 x 4096: 16.7 and 21.9).  fp32's three parts of x leave LDS for
// eight at sixteen entries (13 KB a wave), and fewer entries take eight too: the waves alone decide the order of a
// sum, which is to be the same for every batch.
// More tiles a workgroup share what a block of x costs.  bf16 x: two from four tiles a CU on (32000 x 4096, one
// entry: 14.2 us against 16.7; 11008 x 4096: 7.4 against 7.1); with more than four entries, whose x is four times as
// long, two from one on (8192 x 4096, eight entries: 6.9 against 7.4, four tiles 8.5) and four from two and a half on
// (11008 x 4096, 16 entries: 9.3, two tiles 11.2; 32000 x 4096: 18.6 and 20.8).  fp32 x: two from one tile a CU on
// (one entry, groups of 128: 6144 x 4096 8.8 us, one tile 8.9, four 13.0; 11008 x 4096 12.5, 12.0 and 13.4; 16384 x
// 4096 13.2, 15.3 and 13.8; 32000 x 4096 23.0, 26.6 and 21.8, but groups of 32 25.3, 28.2 and 27.8), with more than
// four entries as for bf16 (16 entries: 8192 x 4096 two tiles 12.6, four 16.0, one 18.5; 11008 x 4096 22.5, 16.3 and
// 26.3; 32000 x 4096 44.7, 32.2 and 67.6; groups of 32 45.2, 34.2 and 69.9).
constexpr int kCUs = 256;
template <int G, typename XT, typename ST>
void w4_shape(const W4Kernel& t, hipStream_t s) {
  const bool many = t.B > 4, one = t.B == 1;
  if constexpr (sizeof(XT) == 2) {
    if (t.tiles <= kCUs) {
      if (many) w4_run<G, XT, ST, 16, 1, 16, 4>(t, s);
      else if (one) w4_run<G, XT, ST, 16, 1, 4, 1>(t, s);
      else w4_run<G, XT, ST, 16, 1, 4, 4>(t, s);
      return;
    }
    if (!many && t.tiles <= 4 * kCUs) {
      if (one) w4_run<G, XT, ST, 8, 1, 4, 1>(t, s);
      else w4_run<G, XT, ST, 8, 1, 4, 4>(t, s);
      return;
    }
  } else if (t.tiles <= kCUs) {
    if (many) w4_run<G, XT, ST, 8, 1, 16, 4>(t, s);
    else w4_run<G, XT, ST, 8, 1, 4, 4>(t, s);
    return;
  }
  if constexpr (sizeof(XT) == 2)
    if (one) return w4_run<G, XT, ST, 8, 2, 4, 1>(t, s);
  if (many && t.tiles > 5 * kCUs / 2) w4_run<G, XT, ST, 8, 4, 16, 4>(t, s);
  else if (many) w4_run<G, XT, ST, 8, 2, 16, 4>(t, s);
  else w4_run<G, XT, ST, 8, 2, 4, 4>(t, s);
}
}  // namespace

size_t w4_bytes(int64_t rows, int64_t cols, int group, int scales_bf16) {
  return (size_t)w4_tiles(rows) * w4_chunks(cols) * w4_block_bytes(group, scales_bf16 ? 2 : 4);
}

hipError_t launch_w4_pack(const uint8_t* codes, const void* scales, int scales_bf16, const uint8_t* zeros, int64_t rows,
                          int64_t cols, int group, uint8_t* packed, hipStream_t s) {
  const int64_t chunks = w4_chunks(cols), words = w4_tiles(rows) * chunks * 256;
  const int64_t groups = (cols + group - 1) / group, count = w4_tiles(rows) * chunks * (kChunk / group) * 16;
  const int bytes = w4_block_bytes(group, scales_bf16 ? 2 : 4);
  hipLaunchKernelGGL(k_w4_codes, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s, codes, rows, cols, chunks, words,
                     bytes, packed);
  const dim3 grid((unsigned)((count + 255) / 256));
  if (scales_bf16)
    hipLaunchKernelGGL((k_w4_scales<uint16_t>), grid, dim3(256), 0, s, static_cast<const uint16_t*>(scales), zeros, rows,
                       groups, chunks, kChunk / group, count, bytes, packed);
  else
    hipLaunchKernelGGL((k_w4_scales<float>), grid, dim3(256), 0, s, static_cast<const float*>(scales), zeros, rows, groups,
                       chunks, kChunk / group, count, bytes, packed);
  return hipGetLastError();
}

hipError_t launch_w4_gemv(const W4Args& a, hipStream_t s) {
  const W4Kernel t{a.packed, a.x, a.y, a.rows, a.cols, w4_chunks(a.cols), w4_tiles(a.rows), a.B, a.y_bf16};
  const auto run = [&](auto run_g) {
    if (a.x_bf16) return a.scales_bf16 ? run_g(uint16_t(), uint16_t()) : run_g(uint16_t(), float());
    return a.scales_bf16 ? run_g(float(), uint16_t()) : run_g(float(), float());
  };
  switch (a.group) {
    case 32: run([&](auto x, auto sc) { w4_shape<32, decltype(x), decltype(sc)>(t, s); }); break;
    case 64: run([&](auto x, auto sc) { w4_shape<64, decltype(x), decltype(sc)>(t, s); }); break;
    default: run([&](auto x, auto sc) { w4_shape<128, decltype(x), decltype(sc)>(t, s); }); break;
  }
  return hipGetLastError();
}

}  // namespace f2i
