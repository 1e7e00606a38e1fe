// C ABI of libfairy2i.so: argument checks, status codes, dispatch to the HIP launchers.
// The operations themselves are specified in include/fairy2i.h.
#include "fairy2i.h"

#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <memory>
#include <mutex>
#include <new>

#include "common.hpp"

namespace {

thread_local char g_err[512] = "";

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return status;
}

int ok() {
  g_err[0] = '\0';
  return FAIRY2I_OK;
}

int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(FAIRY2I_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxRows = int64_t(1) << 28;   // complex rows n
constexpr int64_t kMaxCols = int64_t(1) << 22;   // complex columns m
constexpr int64_t kMaxTokens = int64_t(1) << 20;

int check_stages(int T) {
  if (T < 1 || T > 4) return fail(FAIRY2I_ERR_STAGES, "T = %d, must be in [1, 4]", T);
  return FAIRY2I_OK;
}

// The fp4 GEMV's fp32 sums stay exact integers up to 24 m < 2^24.
constexpr int64_t kMaxColsF4 = int64_t(1) << 19;

int check_f4_cols(int kernel, int64_t m) {
  if (kernel == FAIRY2I_GEMV_MFMA_F4 && m > kMaxColsF4)
    return fail(FAIRY2I_ERR_SHAPE, "m = %lld: the fp4 MFMA GEMV takes m <= %lld", (long long)m,
                (long long)kMaxColsF4);
  return FAIRY2I_OK;
}

int check_nm(int64_t n, int64_t m) {
  if (n < 1 || n > kMaxRows) return fail(FAIRY2I_ERR_SHAPE, "n = %lld out of range", (long long)n);
  if (m < 64 || m > kMaxCols || m % 64 != 0)
    return fail(FAIRY2I_ERR_SHAPE, "m = %lld: need m >= 64 and m %% 64 == 0", (long long)m);
  return FAIRY2I_OK;
}

size_t align16(size_t v) { return (v + 15) & ~size_t(15); }

// Kernels with one 256-thread workgroup per row (quantizers, dequantize) address at most
// 2^24 - 1 workgroups per launch (2^32 work-items).
constexpr int64_t kMaxRowLaunch = (int64_t(1) << 24) - 1;
int check_row_launch(int64_t n) {
  if ((n + 15) / 16 * 16 > kMaxRowLaunch)
    return fail(FAIRY2I_ERR_SHAPE, "n = %lld: one launch covers at most %lld rows", (long long)n,
                (long long)(kMaxRowLaunch / 16 * 16));
  return FAIRY2I_OK;
}

}  // namespace

extern "C" {

int fairy2i_abi_version(void) { return FAIRY2I_ABI_VERSION; }

const char* fairy2i_last_error(void) { return g_err; }

const char* fairy2i_status_string(int status) {
  switch (status) {
    case FAIRY2I_OK: return "ok";
    case FAIRY2I_ERR_NULL: return "null pointer";
    case FAIRY2I_ERR_SHAPE: return "bad shape";
    case FAIRY2I_ERR_STAGES: return "bad stage count";
    case FAIRY2I_ERR_DTYPE: return "bad dtype";
    case FAIRY2I_ERR_ALIGN: return "misaligned pointer";
    case FAIRY2I_ERR_WORKSPACE: return "workspace too small";
    case FAIRY2I_ERR_HIP: return "HIP error";
    default: return "unknown status";
  }
}

static int quantize_any(const void* R, int r_bf16, int64_t two_n, int64_t two_m, int T, uint8_t* packed,
                        float* scales, double* scales64, uint8_t* codes, hipStream_t stream) {
  if (!R || !packed || !scales) return fail(FAIRY2I_ERR_NULL, "R, packed and scales are required");
  if (int s = check_stages(T)) return s;
  if (two_n < 2 || two_n % 2 || two_m < 2 || two_m % 2)
    return fail(FAIRY2I_ERR_SHAPE, "R is %lld x %lld; both sizes must be even",
                (long long)two_n, (long long)two_m);
  const int64_t n = two_n / 2, m = two_m / 2;
  if (int s = check_nm(n, m)) return s;
  if (int s = check_row_launch(n)) return s;
  if (2 * T * m > 65536)
    return fail(FAIRY2I_ERR_SHAPE, "2*T*m = %lld exceeds 65536", (long long)(2 * T * m));
  if (!aligned(R, r_bf16 ? 2 : 4) || !aligned(packed, 16) || !aligned(scales, 4) ||
      (scales64 && !aligned(scales64, 8)) || (codes && !aligned(codes, 16)))
    return fail(FAIRY2I_ERR_ALIGN, "R needs 4 (fp32) or 2 (bf16), scales 4, scales64 8, packed/codes 16-byte alignment");
  return hip_status(f2i::launch_quantize(R, r_bf16, (int)n, (int)m, T, packed, scales, scales64, codes, stream),
                    "quantize launch");
}

int fairy2i_quantize(const float* R, int64_t two_n, int64_t two_m, int T, uint8_t* packed,
                     float* scales, double* scales64, uint8_t* codes, hipStream_t stream) {
  return quantize_any(R, 0, two_n, two_m, T, packed, scales, scales64, codes, stream);
}

int fairy2i_quantize_bf16(const uint16_t* R, int64_t two_n, int64_t two_m, int T, uint8_t* packed,
                          float* scales, double* scales64, uint8_t* codes, hipStream_t stream) {
  return quantize_any(R, 1, two_n, two_m, T, packed, scales, scales64, codes, stream);
}

int fairy2i_quantize_grouped(int count, const void* const* R, int R_dtype, int64_t two_n, int64_t two_m, int T,
                             uint8_t* const* packed, float* const* scales, double* const* scales64,
                             uint8_t* const* codes, hipStream_t stream) {
  if (count < 0) return fail(FAIRY2I_ERR_SHAPE, "count = %d", count);
  if (count > 0 && (!R || !packed || !scales)) return fail(FAIRY2I_ERR_NULL, "R, packed and scales arrays are required");
  if (R_dtype != FAIRY2I_F32 && R_dtype != FAIRY2I_BF16)
    return fail(FAIRY2I_ERR_DTYPE, "R_dtype %d: need F32 or BF16", R_dtype);
  if (int s = check_stages(T)) return s;
  if (two_n < 2 || two_n % 2 || two_m < 2 || two_m % 2)
    return fail(FAIRY2I_ERR_SHAPE, "R is %lld x %lld; both sizes must be even",
                (long long)two_n, (long long)two_m);
  const int64_t n = two_n / 2, m = two_m / 2;
  if (int s = check_nm(n, m)) return s;
  if (2 * T * m > 65536)
    return fail(FAIRY2I_ERR_SHAPE, "2*T*m = %lld exceeds 65536", (long long)(2 * T * m));
  const int64_t rows = (n + 15) / 16 * 16;
  if (std::min(count, f2i::kMaxQuantItems) * rows > kMaxRowLaunch)
    return fail(FAIRY2I_ERR_SHAPE, "%d layers of %lld rows exceed one launch's %lld workgroups",
                std::min(count, f2i::kMaxQuantItems), (long long)rows, (long long)kMaxRowLaunch);
  const int bf16 = R_dtype == FAIRY2I_BF16;
  for (int k = 0; k < count; ++k) {
    if (!R[k] || !packed[k] || !scales[k]) return fail(FAIRY2I_ERR_NULL, "layer %d: R, packed and scales are required", k);
    const double* s64 = scales64 ? scales64[k] : nullptr;
    const uint8_t* cd = codes ? codes[k] : nullptr;
    if (!aligned(R[k], bf16 ? 2 : 4) || !aligned(packed[k], 16) || !aligned(scales[k], 4) ||
        (s64 && !aligned(s64, 8)) || (cd && !aligned(cd, 16)))
      return fail(FAIRY2I_ERR_ALIGN, "layer %d: R needs 4 (fp32) or 2 (bf16), scales 4, scales64 8, "
                  "packed/codes 16-byte alignment", k);
  }
  for (int k0 = 0; k0 < count; k0 += f2i::kMaxQuantItems) {
    f2i::QuantGroup grp;
    grp.count = std::min(count - k0, f2i::kMaxQuantItems);
    for (int k = 0; k < grp.count; ++k)
      grp.items[k] = f2i::QuantItem{R[k0 + k], packed[k0 + k], scales[k0 + k],
                                    scales64 ? scales64[k0 + k] : nullptr, codes ? codes[k0 + k] : nullptr};
    if (int s = hip_status(f2i::launch_quantize_group(grp, bf16, (int)n, (int)m, T, stream), "grouped quantize launch"))
      return s;
  }
  return ok();
}

size_t fairy2i_quantize_tensor_workspace_bytes(int64_t n, int64_t m, int T) {
  (void)m;
  (void)T;
  if (n < 1 || n > kMaxRows) return 0;
  return f2i::quantize_tensor_workspace_bytes(n);
}

int fairy2i_quantize_tensor(const void* R, int R_dtype, int64_t two_n, int64_t two_m, int T,
                            void* workspace, size_t workspace_bytes, uint8_t* packed, float* scales,
                            double* scales64, uint8_t* codes, hipStream_t stream) {
  if (!R || !packed || !scales || !workspace)
    return fail(FAIRY2I_ERR_NULL, "R, workspace, packed and scales are required");
  if (R_dtype != FAIRY2I_F32 && R_dtype != FAIRY2I_BF16)
    return fail(FAIRY2I_ERR_DTYPE, "R_dtype %d: need F32 or BF16", R_dtype);
  if (int s = check_stages(T)) return s;
  if (two_n < 2 || two_n % 2 || two_m < 2 || two_m % 2)
    return fail(FAIRY2I_ERR_SHAPE, "R is %lld x %lld; both sizes must be even",
                (long long)two_n, (long long)two_m);
  const int64_t n = two_n / 2, m = two_m / 2;
  if (int s = check_nm(n, m)) return s;
  if (int s = check_row_launch(n)) return s;
  if (2 * m > 65536) return fail(FAIRY2I_ERR_SHAPE, "m = %lld exceeds 32768", (long long)m);
  const size_t need = f2i::quantize_tensor_workspace_bytes(n);
  if (workspace_bytes < need)
    return fail(FAIRY2I_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace_bytes, need);
  const int bf16 = R_dtype == FAIRY2I_BF16;
  if (!aligned(R, bf16 ? 2 : 4) || !aligned(workspace, 16) || !aligned(packed, 16) || !aligned(scales, 4) ||
      (scales64 && !aligned(scales64, 8)) || (codes && !aligned(codes, 16)))
    return fail(FAIRY2I_ERR_ALIGN, "R needs 4 (fp32) or 2 (bf16), scales 4, scales64 8, workspace/packed/codes 16-byte alignment");
  return hip_status(f2i::launch_quantize_tensor(R, bf16, (int)n, (int)m, T, workspace, packed, scales,
                                                scales64, codes, stream),
                    "per-tensor quantize launch");
}

int fairy2i_pack(const uint8_t* codes, int64_t n, int64_t m, int T, uint8_t* packed,
                 hipStream_t stream) {
  if (!codes || !packed) return fail(FAIRY2I_ERR_NULL, "codes and packed are required");
  if (int s = check_stages(T)) return s;
  if (int s = check_nm(n, m)) return s;
  if (!aligned(codes, 16) || !aligned(packed, 16))
    return fail(FAIRY2I_ERR_ALIGN, "codes and packed need 16-byte alignment");
  return hip_status(f2i::launch_pack(codes, (int)n, (int)m, T, packed, stream), "pack launch");
}

// Checks the dtype / algorithm / batch combination of a GEMV call and resolves AUTO and MFMA to
// the kernel that runs.  Returns minus the status (with the message recorded) on a bad combination.
// The fp4 GEMV on bf16 x builds each row's digit records in LDS (fp4, 16 bytes per record): at
// most 32 chunks of 256 columns over the batch entries (64 KB).  AUTO takes it for launches of at
// least kF4FusedMinTiles tiles, whose workgroups stay resident and build the records once for many
// tiles (those workgroups need one x for the launch).  In smaller launches at batch 1 each wave
// builds the records of its own chunks only; per launch, 32 distinct T = 2 layers in a graph,
// bf16 / fp4 us: m = 2048 16 tiles 5.08 / 5.00, 256 tiles 5.94 / 4.77, 1535 tiles 21.06 / 14.76;
// m = 4096, 5504 and 8192 faster at every size (8192, 1535 tiles: 58.76 / 44.35); m = 1024 16 tiles
// 3.85 / 4.09, 64 tiles 4.11 / 4.11, 128 tiles 4.23 / 4.18, 1535 tiles 12.56 / 10.84; m = 512
// slower up to 128 tiles and at 1535.  At batch 2 the per-tile build and the second batch entry's
// operands make it slower than bf16 at every small size measured (m = 512 to 4096, 16 to 1535
// tiles).
constexpr int kMaxF4FusedColumns = 8192;
constexpr int64_t kF4FusedMinTiles = 1536;
constexpr int64_t kF4FusedSmallMinM = 2048;          // any launch size from here
constexpr int64_t kF4FusedShortMinM = 1024;          // and from kF4FusedShortMinTiles tiles from here
constexpr int64_t kF4FusedShortMinTiles = 128;
static bool f4_records_fit(int64_t m, int64_t B) { return m * B <= kMaxF4FusedColumns; }
static bool f4_fused_small_wins(int64_t B, int64_t m, int64_t tiles) {
  return B == 1 && (m >= kF4FusedSmallMinM || (m >= kF4FusedShortMinM && tiles >= kF4FusedShortMinTiles));
}

// At batch 3-4 the fp4 kernel on x split into two fp8 parts beats the bf16 kernel on large
// launches (1 GiB pools, bf16 / fp4 x fp8 us: 4096 x 4096 at B = 3 337.7 / 262.9, B = 4 316.4 /
// 247.2; 11008 x 4096 B = 4 301.6 / 252.4; 4096 x 11008 B = 4 289.1 / 250.5); at B = 8 the two are
// within 3 % either way and at B = 16 it takes twice as long (its four column groups need four-wave
// workgroups); in the decode step's small launches (4-23 MB) its eight-tile workgroups leave most
// of the chip idle (B = 8: 18.9 against 11.4 us per q/k/v launch).
constexpr int64_t kF4x8MinTiles = 1536;
constexpr int64_t kF4x8MaxM = int64_t(1) << 19;
static bool f4x8_wins(int64_t B, int64_t m, int64_t tiles) {
  return B >= 3 && B <= 4 && tiles >= kF4x8MinTiles && m <= kF4x8MaxM;
}

static int gemv_kernel(int x_dtype, int y_dtype, int algo, int64_t B, int64_t m, int64_t tiles = 0,
                       bool shared_x = true) {
  if (x_dtype != FAIRY2I_F32 && x_dtype != FAIRY2I_BF16 && x_dtype != FAIRY2I_X_DIGITS &&
      x_dtype != FAIRY2I_X_DIGITS_F6)
    return -fail(FAIRY2I_ERR_DTYPE, "x_dtype %d: need F32, BF16, X_DIGITS or X_DIGITS_F6", x_dtype);
  if (y_dtype != FAIRY2I_F32 && y_dtype != FAIRY2I_BF16)
    return -fail(FAIRY2I_ERR_DTYPE, "y_dtype %d: need F32 or BF16", y_dtype);
  if (algo < FAIRY2I_GEMV_AUTO || algo > FAIRY2I_GEMV_MFMA_F4)
    return -fail(FAIRY2I_ERR_DTYPE, "unknown GEMV algorithm %d", algo);
  if (B < 1 || B > 16) return -fail(FAIRY2I_ERR_SHAPE, "B = %lld: need 1 <= B <= 16", (long long)B);
  int kernel = algo;
  if (kernel == FAIRY2I_GEMV_AUTO)
    kernel = x_dtype == FAIRY2I_X_DIGITS    ? FAIRY2I_GEMV_MFMA_I8
           : x_dtype == FAIRY2I_X_DIGITS_F6 ? FAIRY2I_GEMV_MFMA_F4
           : x_dtype == FAIRY2I_BF16        ? ((B <= 2 && f4_records_fit(m, B) &&
                                                        (tiles >= kF4FusedMinTiles ? shared_x
                                                                                   : f4_fused_small_wins(B, m, tiles))) ||
                                                       f4x8_wins(B, m, tiles)
                                                   ? FAIRY2I_GEMV_MFMA_F4 : FAIRY2I_GEMV_MFMA_BF16)
                                            : FAIRY2I_GEMV_VALU;
  if (kernel == FAIRY2I_GEMV_MFMA) kernel = FAIRY2I_GEMV_MFMA_BF16;
  if (kernel == FAIRY2I_GEMV_MFMA_I8) {
    if (x_dtype != FAIRY2I_X_DIGITS)
      return -fail(FAIRY2I_ERR_DTYPE, "the int8 MFMA GEMV takes x in digit form (fairy2i_x_digits)");
    if (B > 2) return -fail(FAIRY2I_ERR_SHAPE, "B = %lld: the int8 MFMA GEMV takes B <= 2", (long long)B);
  } else if (kernel == FAIRY2I_GEMV_MFMA_F4) {
    if (x_dtype != FAIRY2I_X_DIGITS_F6 && x_dtype != FAIRY2I_BF16)
      return -fail(FAIRY2I_ERR_DTYPE, "the fp4 MFMA GEMV takes bf16 x or x in fp6 digit form (fairy2i_x_digits_f6)");
    if (B > 2 && x_dtype != FAIRY2I_BF16)
      return -fail(FAIRY2I_ERR_SHAPE, "B = %lld: the fp4 MFMA GEMV on a digit form takes B <= 2 (bf16 x: B <= 16)",
                   (long long)B);
    if (x_dtype == FAIRY2I_BF16 && B <= 2 && m > 0 && !f4_records_fit(m, B))
      return -fail(FAIRY2I_ERR_SHAPE, "m = %lld, B = %lld: the fp4 MFMA GEMV on bf16 x takes m * B <= %d "
                   "(its digit records are built in LDS); make the digit form with fairy2i_x_digits_f6",
                   (long long)m, (long long)B, kMaxF4FusedColumns);
    if (x_dtype == FAIRY2I_BF16 && B <= 2 && !shared_x && tiles >= kF4FusedMinTiles)
      return -fail(FAIRY2I_ERR_SHAPE, "the fp4 MFMA GEMV on bf16 x needs one x for every item of a launch of "
                   "%lld tiles or more (give the items' x as one digit form, or use the bf16 kernel)",
                   (long long)kF4FusedMinTiles);
  } else if (x_dtype == FAIRY2I_X_DIGITS) {
    return -fail(FAIRY2I_ERR_DTYPE, "x in digit form needs the int8 MFMA GEMV");
  } else if (x_dtype == FAIRY2I_X_DIGITS_F6) {
    return -fail(FAIRY2I_ERR_DTYPE, "x in fp6 digit form needs the fp4 MFMA GEMV");
  } else if (kernel == FAIRY2I_GEMV_MFMA_BF16 && x_dtype != FAIRY2I_BF16) {
    return -fail(FAIRY2I_ERR_DTYPE, "the bf16 MFMA GEMV takes bf16 x only");
  }
  return kernel;
}

size_t fairy2i_packed_bytes(int64_t n, int64_t m, int T) {
  if (n < 1 || m < 1 || T < 1) return 0;
  return (size_t)((n + 15) / 16) * 16 * (size_t)T * 2 * (size_t)(m / 4);
}

size_t fairy2i_x_digits_bytes(int64_t m, int64_t B) {
  if (m < 1 || B < 1) return 0;
  return f2i::x_digits_bytes(m, B);
}

int fairy2i_x_digits(const void* x, int x_dtype, int64_t m, int64_t B, void* digits, hipStream_t stream) {
  if (!x || !digits) return fail(FAIRY2I_ERR_NULL, "x and digits are required");
  if (x_dtype != FAIRY2I_F32 && x_dtype != FAIRY2I_BF16)
    return fail(FAIRY2I_ERR_DTYPE, "x_dtype %d: need F32 or BF16", x_dtype);
  if (m < 64 || m > kMaxCols || m % 64 != 0)
    return fail(FAIRY2I_ERR_SHAPE, "m = %lld: need m >= 64 and m %% 64 == 0", (long long)m);
  if (B < 1 || B > 2) return fail(FAIRY2I_ERR_SHAPE, "B = %lld: the digit form takes 1 <= B <= 2", (long long)B);
  if (!aligned(x, 16) || !aligned(digits, 16))
    return fail(FAIRY2I_ERR_ALIGN, "x and digits need 16-byte alignment");
  return hip_status(f2i::launch_x_digits(x, x_dtype == FAIRY2I_BF16, (int)m, (int)B, digits, stream),
                    "x digits launch");
}

size_t fairy2i_x_digits_f6_bytes(int64_t m, int64_t B) {
  if (m < 1 || B < 1) return 0;
  return f2i::x_digits_f6_bytes(m, B);
}

int fairy2i_x_digits_f6(const void* x, int x_dtype, int64_t m, int64_t B, void* digits, hipStream_t stream) {
  if (!x || !digits) return fail(FAIRY2I_ERR_NULL, "x and digits are required");
  if (x_dtype != FAIRY2I_F32 && x_dtype != FAIRY2I_BF16)
    return fail(FAIRY2I_ERR_DTYPE, "x_dtype %d: need F32 or BF16", x_dtype);
  if (m < 64 || m > kMaxCols || m % 64 != 0)
    return fail(FAIRY2I_ERR_SHAPE, "m = %lld: need m >= 64 and m %% 64 == 0", (long long)m);
  if (B < 1 || B > 2) return fail(FAIRY2I_ERR_SHAPE, "B = %lld: the fp6 digit form takes 1 <= B <= 2", (long long)B);
  if (!aligned(x, 16) || !aligned(digits, 16))
    return fail(FAIRY2I_ERR_ALIGN, "x and digits need 16-byte alignment");
  return hip_status(f2i::launch_x_digits_f6(x, x_dtype == FAIRY2I_BF16, (int)m, (int)B, digits, stream),
                    "x fp6 digits launch");
}

// The fp4 matrix-core GEMVs: batch 1-2 on a digit form or bf16 x (launch_gemv_f4_group); batch 3-16
// on bf16 x split into fp8 parts (launch_gemv_f8x_group).
static hipError_t launch_f4_family(const f2i::GemvGroup& grp, int64_t m, int T, int64_t B, int ybf, int x_dtype,
                                   hipStream_t stream) {
  if (B > 2) return f2i::launch_gemv_f8x_group(grp, (int)m, T, (int)B, ybf, stream);
  return f2i::launch_gemv_f4_group(grp, (int)m, T, (int)B, ybf, x_dtype == FAIRY2I_BF16, stream);
}

int fairy2i_gemv(const uint8_t* packed, const float* scales, int64_t n, int64_t m, int T,
                 const void* x, int x_dtype, int64_t B, void* y, int y_dtype, int algo,
                 hipStream_t stream) {
  if (!packed || !scales || !x || !y) return fail(FAIRY2I_ERR_NULL, "packed, scales, x and y are required");
  const int kernel = gemv_kernel(x_dtype, y_dtype, algo, B, m, (n + 15) / 16);
  if (kernel < 0) return -kernel;
  if (int s = check_stages(T)) return s;
  if (int s = check_nm(n, m)) return s;
  if (int s = check_f4_cols(kernel, m)) return s;
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(scales, 4))
    return fail(FAIRY2I_ERR_ALIGN, "packed, x and y need 16-byte alignment, scales 4");
  if (kernel == FAIRY2I_GEMV_MFMA_F4 && B > 2) {
    f2i::GemvGroup grp;
    grp.count = 1;
    grp.tile_start[0] = 0;
    grp.tile_start[1] = (int)((n + 15) / 16);
    grp.items[0] = f2i::GemvItem{packed, scales, x, y, (int)n};
    return hip_status(launch_f4_family(grp, m, T, B, y_dtype == FAIRY2I_BF16, x_dtype, stream),
                      "gemv (fp4 x fp8 mfma) launch");
  }
  if (kernel == FAIRY2I_GEMV_MFMA_F4)
    return hip_status(f2i::launch_gemv_f4(packed, scales, (int)n, (int)m, T, x, (int)B, y,
                                          y_dtype == FAIRY2I_BF16, x_dtype == FAIRY2I_BF16, stream),
                      "gemv (fp4 mfma) launch");
  if (kernel == FAIRY2I_GEMV_MFMA_I8)
    return hip_status(f2i::launch_gemv_i8(packed, scales, (int)n, (int)m, T, x, (int)B, y,
                                          y_dtype == FAIRY2I_BF16, stream),
                      "gemv (int8 mfma) launch");
  if (kernel == FAIRY2I_GEMV_MFMA_BF16)
    return hip_status(f2i::launch_gemv_mfma(packed, scales, (int)n, (int)m, T, x, (int)B, y,
                                            y_dtype == FAIRY2I_BF16, nullptr, stream),
                      "gemv (bf16 mfma) launch");
  return hip_status(f2i::launch_gemv_valu(packed, scales, (int)n, (int)m, T, x,
                                          x_dtype == FAIRY2I_BF16, (int)B, y,
                                          y_dtype == FAIRY2I_BF16, stream),
                    "gemv (valu) launch");
}

int fairy2i_gemv_grouped(const fairy2i_gemv_item* items, int count, int64_t m, int T, int x_dtype,
                         int64_t B, int y_dtype, int algo, hipStream_t stream) {
  if (!items) return fail(FAIRY2I_ERR_NULL, "items is required");
  if (count < 1) return fail(FAIRY2I_ERR_SHAPE, "count = %d: need at least one item", count);
  for (int k = 0; k < count; ++k)
    if (!items[k].packed || !items[k].scales || !items[k].x || !items[k].y)
      return fail(FAIRY2I_ERR_NULL, "item %d: packed, scales, x and y are required", k);
  int64_t all_tiles = 0;
  bool shared_x = true;
  for (int k = 0; k < count; ++k) {
    all_tiles += (items[k].n + 15) / 16;
    shared_x = shared_x && items[k].x == items[0].x;
  }
  const int kernel = gemv_kernel(x_dtype, y_dtype, algo, B, m, all_tiles, shared_x);
  if (kernel < 0) return -kernel;
  if (int s = check_stages(T)) return s;
  for (int k = 0; k < count; ++k)
    if (int s = check_nm(items[k].n, m)) return s;
  if (int s = check_f4_cols(kernel, m)) return s;
  for (int k = 0; k < count; ++k)
    if (!aligned(items[k].packed, 16) || !aligned(items[k].x, 16) || !aligned(items[k].y, 16) ||
        !aligned(items[k].scales, 4))
      return fail(FAIRY2I_ERR_ALIGN, "item %d: packed, x and y need 16-byte alignment, scales 4", k);
  if (kernel == FAIRY2I_GEMV_VALU) {
    for (int k = 0; k < count; ++k) {
      const fairy2i_gemv_item& it = items[k];
      int s = fairy2i_gemv(it.packed, it.scales, it.n, m, T, it.x, x_dtype, B, it.y, y_dtype, algo, stream);
      if (s != FAIRY2I_OK) return s;
    }
    return ok();
  }
  for (int k0 = 0; k0 < count; k0 += f2i::kMaxGroup) {
    f2i::GemvGroup grp;
    grp.count = count - k0 < f2i::kMaxGroup ? count - k0 : f2i::kMaxGroup;
    int tiles = 0;
    for (int k = 0; k < grp.count; ++k) {
      const fairy2i_gemv_item& it = items[k0 + k];
      grp.tile_start[k] = tiles;
      grp.items[k] = f2i::GemvItem{it.packed, it.scales, it.x, it.y, (int)it.n};
      tiles += (int)((it.n + 15) / 16);
    }
    grp.tile_start[grp.count] = tiles;
    const int ybf = y_dtype == FAIRY2I_BF16;
    hipError_t e = kernel == FAIRY2I_GEMV_MFMA_F4
                       ? launch_f4_family(grp, m, T, B, ybf, x_dtype, stream)
                 : kernel == FAIRY2I_GEMV_MFMA_I8 ? f2i::launch_gemv_i8_group(grp, (int)m, T, (int)B, ybf, stream)
                 : f2i::launch_gemv_mfma_group(grp, (int)m, T, (int)B, ybf, stream);
    if (e != hipSuccess) return hip_status(e, "gemv (grouped mfma) launch");
  }
  return ok();
}

int fairy2i_gemv_strided(const uint8_t* packed, int64_t packed_stride, const float* scales,
                         int64_t scales_stride, int64_t n, int64_t m, int T, const void* x,
                         int x_dtype, int64_t B, void* y, int64_t y_stride, int y_dtype,
                         int64_t batch, int algo, hipStream_t stream) {
  if (!packed || !scales || !x || !y) return fail(FAIRY2I_ERR_NULL, "packed, scales, x and y are required");
  const int kernel = gemv_kernel(x_dtype, y_dtype, algo, B, m, batch > 0 && n > 0 ? batch * ((n + 15) / 16) : 0);
  if (kernel < 0) return -kernel;
  if (int s = check_stages(T)) return s;
  if (int s = check_nm(n, m)) return s;
  if (int s = check_f4_cols(kernel, m)) return s;
  const int64_t tiles = (n + 15) / 16;
  if (batch < 1 || batch > (int64_t(1) << 30) / tiles)
    return fail(FAIRY2I_ERR_SHAPE, "batch = %lld: need 1 <= batch and batch * ceil(n/16) <= 2^30", (long long)batch);
  const int64_t y_elem = y_dtype == FAIRY2I_BF16 ? 2 : 4;
  if (packed_stride < 0 || scales_stride < 0 || y_stride < 0)
    return fail(FAIRY2I_ERR_SHAPE, "strides must be >= 0");
  if (batch > 1 && y_stride < 2 * n * B)
    return fail(FAIRY2I_ERR_SHAPE, "y_stride = %lld: outputs of different matrices overlap (need >= 2nB = %lld)",
                (long long)y_stride, (long long)(2 * n * B));
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(scales, 4) ||
      packed_stride % 16 != 0 || (y_stride * y_elem) % 16 != 0)
    return fail(FAIRY2I_ERR_ALIGN, "packed, x and y (and their strides) need 16-byte alignment, scales 4");
  if (kernel == FAIRY2I_GEMV_VALU) {
    for (int64_t k = 0; k < batch; ++k) {
      int s = fairy2i_gemv(packed + k * packed_stride, scales + k * scales_stride, n, m, T, x, x_dtype, B,
                           static_cast<uint8_t*>(y) + k * y_stride * y_elem, y_dtype, algo, stream);
      if (s != FAIRY2I_OK) return s;
    }
    return ok();
  }
  f2i::GemvGroup grp;
  grp.count = 1;
  grp.tile_start[0] = 0;
  grp.tile_start[1] = (int)tiles;
  grp.items[0] = f2i::GemvItem{packed, scales, x, y, (int)n};
  grp.batch = (int)batch;
  grp.tiles_per_item = (int)tiles;
  grp.packed_stride = packed_stride;
  grp.scales_stride = scales_stride;
  grp.y_stride = y_stride;
  const int ybf = y_dtype == FAIRY2I_BF16;
  hipError_t e = kernel == FAIRY2I_GEMV_MFMA_F4
                     ? launch_f4_family(grp, m, T, B, ybf, x_dtype, stream)
               : kernel == FAIRY2I_GEMV_MFMA_I8 ? f2i::launch_gemv_i8_group(grp, (int)m, T, (int)B, ybf, stream)
               : f2i::launch_gemv_mfma_group(grp, (int)m, T, (int)B, ybf, stream);
  return hip_status(e, "gemv (strided batch) launch");
}

int fairy2i_dequantize(const uint8_t* packed, const float* scales, int64_t n, int64_t m, int T,
                       void* R, int R_dtype, hipStream_t stream) {
  if (!packed || !scales || !R) return fail(FAIRY2I_ERR_NULL, "packed, scales and R are required");
  if (R_dtype != FAIRY2I_F32 && R_dtype != FAIRY2I_BF16)
    return fail(FAIRY2I_ERR_DTYPE, "R_dtype %d: need F32 or BF16", R_dtype);
  if (int s = check_stages(T)) return s;
  if (int s = check_nm(n, m)) return s;
  if (int s = check_row_launch(n)) return s;
  if (!aligned(packed, 16) || !aligned(R, 16) || !aligned(scales, 4))
    return fail(FAIRY2I_ERR_ALIGN, "packed and R need 16-byte alignment, scales 4");
  return hip_status(f2i::launch_dequant(packed, scales, (int)n, (int)m, T, R, R_dtype == FAIRY2I_BF16, stream),
                    "dequantize launch");
}

int fairy2i_act_quant(const void* x, int x_dtype, int64_t N, int64_t two_m, int8_t* q,
                      float* delta, hipStream_t stream) {
  if (!x || !q || !delta) return fail(FAIRY2I_ERR_NULL, "x, q and delta are required");
  if (x_dtype != FAIRY2I_F32 && x_dtype != FAIRY2I_BF16)
    return fail(FAIRY2I_ERR_DTYPE, "x_dtype %d: need F32 or BF16", x_dtype);
  if (N < 1 || N > kMaxTokens) return fail(FAIRY2I_ERR_SHAPE, "N = %lld out of range", (long long)N);
  if (two_m < 8 || two_m % 8 || two_m > 2 * kMaxCols)
    return fail(FAIRY2I_ERR_SHAPE, "row length %lld: need a positive multiple of 8", (long long)two_m);
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(delta, 4))
    return fail(FAIRY2I_ERR_ALIGN, "x and q need 16-byte alignment, delta 4");
  return hip_status(f2i::launch_act_quant(x, x_dtype == FAIRY2I_BF16, (int)N, (int)two_m, q, delta, stream),
                    "act_quant launch");
}

size_t fairy2i_gemm_workspace_bytes(int64_t n, int64_t m, int T, int64_t N, int x_dtype) {
  (void)n;
  (void)T;
  if (x_dtype == FAIRY2I_I8 || N < 1 || m < 1) return 0;
  return align16((size_t)N * 2 * (size_t)m) + align16((size_t)N * 4);
}

}  // extern "C"

// Argument checks of the prefill GEMM (null -> dtype -> stages -> shape -> alignment), shared by
// fairy2i_gemm and fairy2i_gemm_noalloc.
static int check_gemm(const uint8_t* packed, const float* scales, int64_t n, int64_t m, int T, const void* x,
                      int x_dtype, const float* x_scale, int64_t N, const void* y, int y_dtype) {
  if (!packed || !scales || !x || !y) return fail(FAIRY2I_ERR_NULL, "packed, scales, x and y are required");
  if (x_dtype == FAIRY2I_I8 && !x_scale)
    return fail(FAIRY2I_ERR_NULL, "x_scale (delta) is required with int8 x");
  if (x_dtype != FAIRY2I_F32 && x_dtype != FAIRY2I_BF16 && x_dtype != FAIRY2I_I8)
    return fail(FAIRY2I_ERR_DTYPE, "x_dtype %d: need F32, BF16 or I8", x_dtype);
  if (y_dtype != FAIRY2I_F32 && y_dtype != FAIRY2I_BF16 && y_dtype != FAIRY2I_I32)
    return fail(FAIRY2I_ERR_DTYPE, "y_dtype %d: need F32, BF16 or I32", y_dtype);
  if (int s = check_stages(T)) return s;
  if (int s = check_nm(n, m)) return s;
  if (N < 1 || N > kMaxTokens) return fail(FAIRY2I_ERR_SHAPE, "N = %lld out of range", (long long)N);
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(scales, 4) ||
      (x_scale && !aligned(x_scale, 4)))
    return fail(FAIRY2I_ERR_ALIGN, "packed, x, y, workspace need 16-byte alignment; scales, x_scale 4");
  return FAIRY2I_OK;
}

// The prefill GEMM's launches, with the activation workspace (int8 q, then delta) at `workspace`.
static int gemm_launch(const uint8_t* packed, const float* scales, int64_t n, int64_t m, int T, const void* x,
                       int x_dtype, float* x_scale, int64_t N, void* y, int y_dtype, void* workspace,
                       hipStream_t stream) {
  const int8_t* q = static_cast<const int8_t*>(x);
  const float* delta = x_scale;
  if (x_dtype != FAIRY2I_I8) {
    int8_t* qw = static_cast<int8_t*>(workspace);
    float* dw = x_scale ? x_scale
                        : reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                                   align16((size_t)N * 2 * (size_t)m));
    hipError_t e = f2i::launch_act_quant(x, x_dtype == FAIRY2I_BF16, (int)N, (int)(2 * m), qw, dw, stream);
    if (e != hipSuccess) return hip_status(e, "act_quant launch");
    q = qw;
    delta = dw;
  }
  const int mode = y_dtype == FAIRY2I_F32 ? 0 : (y_dtype == FAIRY2I_BF16 ? 1 : 2);
  return hip_status(f2i::launch_gemm(packed, scales, (int)n, (int)m, T, q, delta, (int)N, y, mode, stream),
                    "gemm launch");
}

// ---- the entry point that allocates nothing: its activation workspace is a static device array ----
//
// `scratch` is one array per GPU, reserved when the library's code object is loaded on that GPU and
// held until the process ends.  In host code its name stands for no device address: the address
// on the current device comes from hipGetSymbolAddress, taken once per device on the entry point's
// first call there and kept in g_scratch_ptr.
constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;
static __device__ __align__(256) uint8_t scratch[kNoAllocScratchBytes];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// Device address of the current device's scratch (looked up once per device).
int scratch_on_current_device(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(e, "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(FAIRY2I_ERR_HIP, "device %d: at most %d devices", dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return hip_status(e, "hipGetSymbolAddress(scratch)");
    if (!p) return fail(FAIRY2I_ERR_HIP, "hipGetSymbolAddress(scratch) returned NULL");
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return FAIRY2I_OK;
}
}  // namespace

extern "C" {

size_t fairy2i_gemm_noalloc_max_bytes(void) { return kNoAllocScratchBytes; }

int fairy2i_gemm_noalloc(const uint8_t* packed, const float* scales, int64_t n, int64_t m, int T,
                         const void* x, int x_dtype, float* x_scale, int64_t N, void* y, int y_dtype,
                         hipStream_t stream) {
  if (int s = check_gemm(packed, scales, n, m, T, x, x_dtype, x_scale, N, y, y_dtype)) return s;
  const size_t need = fairy2i_gemm_workspace_bytes(n, m, T, N, x_dtype);
  if (need > kNoAllocScratchBytes)
    return fail(FAIRY2I_ERR_WORKSPACE,
                "N = %lld tokens of 2m = %lld need %zu bytes of activation workspace; the static scratch "
                "holds %zu (use fairy2i_gemm with a caller workspace)",
                (long long)N, (long long)(2 * m), need, kNoAllocScratchBytes);
  void* ws = nullptr;
  if (need > 0) {
    if (int s = scratch_on_current_device(&ws)) return s;
  }
  return gemm_launch(packed, scales, n, m, T, x, x_dtype, x_scale, N, y, y_dtype, ws, stream);
}

int fairy2i_gemm(const uint8_t* packed, const float* scales, int64_t n, int64_t m, int T,
                 const void* x, int x_dtype, float* x_scale, int64_t N, void* y, int y_dtype,
                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (int s = check_gemm(packed, scales, n, m, T, x, x_dtype, x_scale, N, y, y_dtype)) return s;
  if (workspace && !aligned(workspace, 16))
    return fail(FAIRY2I_ERR_ALIGN, "packed, x, y, workspace need 16-byte alignment; scales, x_scale 4");
  const size_t need = fairy2i_gemm_workspace_bytes(n, m, T, N, x_dtype);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(FAIRY2I_ERR_WORKSPACE, "GEMM needs %zu workspace bytes, got %zu", need,
                workspace ? workspace_bytes : size_t(0));
  return gemm_launch(packed, scales, n, m, T, x, x_dtype, x_scale, N, y, y_dtype, workspace, stream);
}

}  // extern "C"

// ---- low-rank adapters, vocabulary loss, gradient clipping ----

namespace {

// Launch geometry bounds of the adapter kernels: 256 outputs (32 transposed rows) per workgroup in a
// grid dimension of at most 65535.
constexpr int64_t kMaxLoraSide = int64_t(1) << 20;
constexpr int64_t kMaxAdapters = 4096;
constexpr int64_t kMaxSegments = int64_t(1) << 20;

int check_float_dtype(int dtype, const char* name) {
  if (dtype != FAIRY2I_F32 && dtype != FAIRY2I_BF16)
    return fail(FAIRY2I_ERR_DTYPE, "%s %d: need F32 or BF16", name, dtype);
  return FAIRY2I_OK;
}

int check_workspace(const void* workspace, size_t have, size_t need) {
  if (need > 0 && (!workspace || have < need))
    return fail(FAIRY2I_ERR_WORKSPACE, "workspace of %zu bytes, need %zu", workspace ? have : size_t(0), need);
  if (workspace && !aligned(workspace, 16)) return fail(FAIRY2I_ERR_ALIGN, "workspace needs 16-byte alignment");
  return FAIRY2I_OK;
}

// Whether two ranges of device memory share bytes (a NULL one shares none).
bool overlap(const void* p, uint64_t p_bytes, const void* q, uint64_t q_bytes) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + q_bytes && b < a + p_bytes;
}

// A range of device memory that clipping reads or writes.
struct Span {
  uint64_t lo, hi;
  bool written;
};
// Whether a written range shares bytes with any other range.
bool written_twice(Span* spans, int64_t count) {
  std::sort(spans, spans + count, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uint64_t read = 0, written = 0;                // where the ranges up to here end
  for (int64_t k = 0; k < count; ++k) {
    const Span& s = spans[k];
    if (s.lo < written || (s.written && s.lo < read)) return true;
    (s.written ? written : read) = std::max(s.written ? written : read, s.hi);
  }
  return false;
}

int check_lora_n(int64_t n) {
  if (n < 1 || n > kMaxLoraSide) return fail(FAIRY2I_ERR_SHAPE, "n = %lld out of range", (long long)n);
  return FAIRY2I_OK;
}

bool lora_sizes_ok(int64_t N, int64_t m, int64_t r, int64_t S) {
  return N >= 1 && N <= kMaxTokens && m >= 64 && m <= kMaxLoraSide && m % 64 == 0 && r >= 1 && r <= f2i::kMaxLoraRank &&
         S >= 1 && S <= kMaxSegments;
}

int check_lora_sizes(int64_t N, int64_t m, int64_t L, int r, int64_t S) {
  if (N < 1 || N > kMaxTokens) return fail(FAIRY2I_ERR_SHAPE, "N = %lld out of range", (long long)N);
  if (m < 64 || m > kMaxLoraSide || m % 64 != 0)
    return fail(FAIRY2I_ERR_SHAPE, "m = %lld: need 64 <= m <= %lld and m %% 64 == 0", (long long)m, (long long)kMaxLoraSide);
  if (L < 1 || L > kMaxAdapters) return fail(FAIRY2I_ERR_SHAPE, "L = %lld: need 1 <= L <= %lld adapters", (long long)L, (long long)kMaxAdapters);
  if (r < 1 || r > f2i::kMaxLoraRank) return fail(FAIRY2I_ERR_SHAPE, "r = %d: need 1 <= r <= %d", r, f2i::kMaxLoraRank);
  if (S < 1 || S > kMaxSegments) return fail(FAIRY2I_ERR_SHAPE, "S = %lld: need 1 <= S <= %lld segments", (long long)S, (long long)kMaxSegments);
  return FAIRY2I_OK;
}

}  // namespace

extern "C" {

size_t fairy2i_lora_workspace_bytes(int count, int64_t N, int64_t m, int r, int64_t S) {
  if (count < 1 || !lora_sizes_ok(N, m, r, S)) return 0;
  return f2i::lora_workspace_bytes(count, N, m, r, S);
}

int fairy2i_lora_grouped(const fairy2i_lora_item* items, int count, const void* x, int x_dtype, int64_t N, int64_t m,
                         int64_t L, int r, const int32_t* seg_start, const int32_t* seg_adapter, int64_t S, int y_dtype,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!items || !x || !seg_start || !seg_adapter)
    return fail(FAIRY2I_ERR_NULL, "items, x, seg_start and seg_adapter are required");
  if (count < 1) return fail(FAIRY2I_ERR_SHAPE, "count = %d: need at least one item", count);
  for (int k = 0; k < count; ++k)
    if (!items[k].A || !items[k].B || !items[k].alpha || !items[k].base || !items[k].y)
      return fail(FAIRY2I_ERR_NULL, "item %d: A, B, alpha, base and y are required", k);
  if (int s = check_float_dtype(x_dtype, "x_dtype")) return s;
  if (int s = check_float_dtype(y_dtype, "y_dtype")) return s;
  if (int s = check_lora_sizes(N, m, L, r, S)) return s;
  for (int k = 0; k < count; ++k)
    if (int s = check_lora_n(items[k].n)) return s;
  if (!aligned(x, 16) || !aligned(seg_start, 4) || !aligned(seg_adapter, 4))
    return fail(FAIRY2I_ERR_ALIGN, "x needs 16-byte alignment, seg_start and seg_adapter 4");
  for (int k = 0; k < count; ++k)
    if (!aligned(items[k].A, 16) || !aligned(items[k].B, 16) || !aligned(items[k].base, 16) || !aligned(items[k].y, 16) ||
        !aligned(items[k].alpha, 4))
      return fail(FAIRY2I_ERR_ALIGN, "item %d: A, B, base and y need 16-byte alignment, alpha 4", k);
  // every item's y is written while the others' inputs, and all adapters and segments, are read
  const uint64_t ye = y_dtype == FAIRY2I_BF16 ? 2 : 4, xe = x_dtype == FAIRY2I_BF16 ? 2 : 4;
  for (int k = 0; k < count; ++k) {
    const void* y = items[k].y;
    const uint64_t yb = (uint64_t)N * 2 * items[k].n * ye;
    if (overlap(y, yb, x, (uint64_t)N * 2 * m * xe) || (y != items[k].base && overlap(y, yb, items[k].base, yb)))
      return fail(FAIRY2I_ERR_SHAPE, "item %d: y overlaps x, or base without being base", k);
    if (overlap(y, yb, seg_start, (uint64_t)(S + 1) * 4) || overlap(y, yb, seg_adapter, (uint64_t)S * 4))
      return fail(FAIRY2I_ERR_SHAPE, "item %d: y overlaps seg_start or seg_adapter", k);
    for (int j = 0; j < count; ++j) {
      const uint64_t ob = (uint64_t)N * 2 * items[j].n * ye;
      if (j != k && (overlap(y, yb, items[j].y, ob) || overlap(y, yb, items[j].base, ob)))
        return fail(FAIRY2I_ERR_SHAPE, "y of item %d overlaps y or base of item %d", k, j);
      if (overlap(y, yb, items[j].A, (uint64_t)L * r * 2 * m * xe) ||
          overlap(y, yb, items[j].B, (uint64_t)L * 2 * items[j].n * r * xe) || overlap(y, yb, items[j].alpha, (uint64_t)L * 4))
        return fail(FAIRY2I_ERR_SHAPE, "y of item %d overlaps A, B or alpha of item %d", k, j);
    }
  }
  if (int s = check_workspace(workspace, workspace_bytes, f2i::lora_workspace_bytes(count, N, m, r, S))) return s;
  const f2i::LoraArgs args{x, x_dtype == FAIRY2I_BF16, y_dtype == FAIRY2I_BF16, (int)N, (int)S, (int)L, r, m,
                           seg_start, seg_adapter, workspace};
  for (int k0 = 0; k0 < count; k0 += f2i::kMaxLoraItems) {
    f2i::LoraItem grp[f2i::kMaxLoraItems];
    const int num = std::min(count - k0, f2i::kMaxLoraItems);
    for (int k = 0; k < num; ++k) {
      const fairy2i_lora_item& it = items[k0 + k];
      grp[k] = f2i::LoraItem{it.A, it.B, it.alpha, it.base, it.y, it.n};
    }
    const hipError_t e = f2i::launch_lora(args, grp, num, stream);
    if (e != hipSuccess) return hip_status(e, "lora launch");
  }
  return ok();
}

int fairy2i_lora(const void* x, int x_dtype, int64_t N, int64_t m, const void* A, const void* B, const float* alpha,
                 int64_t L, int r, int64_t n, const int32_t* seg_start, const int32_t* seg_adapter, int64_t S,
                 const void* base, void* y, int y_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const fairy2i_lora_item it{A, B, alpha, base, y, n};
  return fairy2i_lora_grouped(&it, 1, x, x_dtype, N, m, L, r, seg_start, seg_adapter, S, y_dtype, workspace,
                              workspace_bytes, stream);
}

size_t fairy2i_lora_backward_workspace_bytes(int64_t N, int64_t m, int64_t n, int64_t L, int r, int64_t S, int x_dtype) {
  if (!lora_sizes_ok(N, m, r, S) || n < 1 || n > kMaxLoraSide || L < 1 || L > kMaxAdapters) return 0;
  return f2i::lora_backward_workspace_bytes(N, m, n, r, (int)L, S, x_dtype == FAIRY2I_BF16);
}

int fairy2i_lora_backward(const void* dy, const void* x, int x_dtype, int64_t N, int64_t m, const void* A, const void* B,
                          const float* alpha, int64_t L, int r, int64_t n, const int32_t* seg_start,
                          const int32_t* seg_adapter, int64_t S, const void* dx_base, void* dx, int dx_dtype, float* dA,
                          float* dB, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!dy || !x || !A || !B || !alpha || !seg_start || !seg_adapter || !dA || !dB)
    return fail(FAIRY2I_ERR_NULL, "dy, x, A, B, alpha, seg_start, seg_adapter, dA and dB are required");
  if (!dx != !dx_base) return fail(FAIRY2I_ERR_NULL, "dx and dx_base go together");
  if (int s = check_float_dtype(x_dtype, "x_dtype")) return s;
  if (dx)
    if (int s = check_float_dtype(dx_dtype, "dx_dtype")) return s;
  if (int s = check_lora_sizes(N, m, L, r, S)) return s;
  if (int s = check_lora_n(n)) return s;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(dx, 16) ||
      !aligned(dx_base, 16) || !aligned(dA, 16) || !aligned(dB, 16) || !aligned(alpha, 4) || !aligned(seg_start, 4) ||
      !aligned(seg_adapter, 4))
    return fail(FAIRY2I_ERR_ALIGN, "dy, x, A, B, dx_base, dx, dA and dB need 16-byte alignment, alpha and the segments 4");
  const uint64_t xe = x_dtype == FAIRY2I_BF16 ? 2 : 4, de = dx_dtype == FAIRY2I_BF16 ? 2 : 4;
  const uint64_t dx_bytes = (uint64_t)N * 2 * m * de;
  if (dx != dx_base && overlap(dx, dx_bytes, dx_base, dx_bytes))
    return fail(FAIRY2I_ERR_SHAPE, "dx overlaps dx_base without being dx_base");
  // dA, dB and dx are written while the other gradients' inputs are read (dx and dx_base: above)
  const struct { const void* p; uint64_t bytes; const char* name; } all[] = {
      {dA, (uint64_t)L * r * 2 * m * 4, "dA"}, {dB, (uint64_t)L * 2 * n * r * 4, "dB"}, {dx, dx_bytes, "dx"},
      {A, (uint64_t)L * r * 2 * m * xe, "A"}, {B, (uint64_t)L * 2 * n * r * xe, "B"}, {alpha, (uint64_t)L * 4, "alpha"},
      {seg_start, (uint64_t)(S + 1) * 4, "seg_start"}, {seg_adapter, (uint64_t)S * 4, "seg_adapter"},
      {x, (uint64_t)N * 2 * m * xe, "x"}, {dy, (uint64_t)N * 2 * n * xe, "dy"}, {dx_base, dx_bytes, "dx_base"}};
  for (int k = 0; k < 3; ++k)
    for (int j = k + 1; j < (k == 2 ? 10 : 11); ++j)
      if (overlap(all[k].p, all[k].bytes, all[j].p, all[j].bytes))
        return fail(FAIRY2I_ERR_SHAPE, "%s overlaps %s", all[k].name, all[j].name);
  if (int s = check_workspace(workspace, workspace_bytes,
                              f2i::lora_backward_workspace_bytes(N, m, n, r, (int)L, S, x_dtype == FAIRY2I_BF16)))
    return s;
  const f2i::LoraBackwardArgs args{dy, x, A, B, alpha, dx_base, dx, dA, dB, x_dtype == FAIRY2I_BF16,
                                   dx_dtype == FAIRY2I_BF16, (int)N, (int)S, (int)L, r, m, n, seg_start, seg_adapter,
                                   workspace};
  return hip_status(f2i::launch_lora_backward(args, stream), "lora backward launch");
}

// N V bounds the tiles of one launch (2^32 work-items at the smallest tile).
static bool vocab_sizes_ok(int64_t N, int64_t V, int64_t K) {
  return N >= 1 && N <= kMaxTokens && V >= 1 && V <= (int64_t(1) << 24) && N * V <= (int64_t(1) << 36) && K >= 64 &&
         K <= 65536 && K % 64 == 0;
}

static int check_vocab_sizes(int64_t N, int64_t V, int64_t K) {
  if (vocab_sizes_ok(N, V, K)) return FAIRY2I_OK;
  return fail(FAIRY2I_ERR_SHAPE, "N = %lld, V = %lld, K = %lld: need 1 <= N <= 2^20, 1 <= V <= 2^24, N V <= 2^36, "
              "64 <= K <= 65536 and K %% 64 == 0", (long long)N, (long long)V, (long long)K);
}

size_t fairy2i_vocab_loss_workspace_bytes(int64_t N, int64_t V, int64_t K, int x_dtype) {
  return vocab_sizes_ok(N, V, K) ? f2i::vocab_loss_workspace_bytes(N, V, K, x_dtype == FAIRY2I_BF16, 0) : 0;
}

int fairy2i_vocab_loss(const void* h, const void* W, int x_dtype, int64_t N, int64_t V, int64_t K, const int64_t* target,
                       float* loss, float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!h || !W || !target || !loss || !lse) return fail(FAIRY2I_ERR_NULL, "h, W, target, loss and lse are required");
  if (int s = check_float_dtype(x_dtype, "x_dtype")) return s;
  if (int s = check_vocab_sizes(N, V, K)) return s;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4))
    return fail(FAIRY2I_ERR_ALIGN, "h and W need 16-byte alignment, target 8, loss and lse 4");
  const uint64_t xe = x_dtype == FAIRY2I_BF16 ? 2 : 4, ob = (uint64_t)N * 4;
  if (overlap(loss, ob, lse, ob) || overlap(loss, ob, target, (uint64_t)N * 8) || overlap(lse, ob, target, (uint64_t)N * 8) ||
      overlap(loss, ob, h, (uint64_t)N * K * xe) || overlap(lse, ob, h, (uint64_t)N * K * xe) ||
      overlap(loss, ob, W, (uint64_t)V * K * xe) || overlap(lse, ob, W, (uint64_t)V * K * xe))
    return fail(FAIRY2I_ERR_SHAPE, "loss and lse must not overlap h, W, target or each other");
  if (int s = check_workspace(workspace, workspace_bytes, fairy2i_vocab_loss_workspace_bytes(N, V, K, x_dtype))) return s;
  f2i::VocabArgs a{};
  a.h = h; a.W = W; a.target = target; a.N = N; a.V = V; a.K = K; a.bf16 = x_dtype == FAIRY2I_BF16;
  a.loss = loss; a.lse_out = lse; a.ws = workspace;
  return hip_status(f2i::launch_vocab_loss(a, stream), "vocabulary loss launch");
}

size_t fairy2i_vocab_loss_backward_workspace_bytes(int64_t N, int64_t V, int64_t K, int x_dtype) {
  return vocab_sizes_ok(N, V, K) ? f2i::vocab_loss_backward_workspace_bytes(N, V, K, x_dtype == FAIRY2I_BF16, 0) : 0;
}

int fairy2i_vocab_loss_backward(const void* h, const void* W, int x_dtype, int64_t N, int64_t V, int64_t K,
                                const int64_t* target, const float* lse, const float* g, void* dh, void* dW,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!h || !W || !target || !lse || !g) return fail(FAIRY2I_ERR_NULL, "h, W, target, lse and g are required");
  if (!dh && !dW) return fail(FAIRY2I_ERR_NULL, "one of dh and dW is required");
  if (int s = check_float_dtype(x_dtype, "x_dtype")) return s;
  if (int s = check_vocab_sizes(N, V, K)) return s;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(dh, 16) || !aligned(dW, 16) || !aligned(target, 8) ||
      !aligned(lse, 4) || !aligned(g, 4))
    return fail(FAIRY2I_ERR_ALIGN, "h, W, dh and dW need 16-byte alignment, target 8, lse and g 4");
  // a piece's dW is stored before the next piece reads the inputs again
  const uint64_t xe = x_dtype == FAIRY2I_BF16 ? 2 : 4, hb = (uint64_t)N * K * xe, wb = (uint64_t)V * K * xe;
  const struct { const void* p; uint64_t bytes; } in[] = {
      {h, hb}, {W, wb}, {target, (uint64_t)N * 8}, {lse, (uint64_t)N * 4}, {g, (uint64_t)N * 4}};
  for (const auto& r : in)
    if (overlap(dh, hb, r.p, r.bytes) || overlap(dW, wb, r.p, r.bytes))
      return fail(FAIRY2I_ERR_SHAPE, "dh and dW must not overlap h, W, target, lse or g");
  if (overlap(dh, hb, dW, wb)) return fail(FAIRY2I_ERR_SHAPE, "dh and dW must not overlap each other");
  if (int s = check_workspace(workspace, workspace_bytes, fairy2i_vocab_loss_backward_workspace_bytes(N, V, K, x_dtype)))
    return s;
  f2i::VocabArgs a{};
  a.h = h; a.W = W; a.target = target; a.N = N; a.V = V; a.K = K; a.bf16 = x_dtype == FAIRY2I_BF16;
  a.lse = lse; a.g = g; a.dh = dh; a.dW = dW; a.ws = workspace;
  return hip_status(f2i::launch_vocab_loss_backward(a, stream), "vocabulary loss backward launch");
}

// ---- verification of drafted tokens ----

// S pieces bounds the workgroups of one launch; a wave looks at a sequence's drafts, one a lane.
static bool verify_sizes_ok(int64_t S, int64_t D, int64_t V) {
  return S >= 1 && S <= kMaxTokens && D >= 1 && D <= 63 && V >= 1 && V <= (int64_t(1) << 24) &&
         S * ((V + 4095) / 4096) <= (int64_t(1) << 23);
}

size_t fairy2i_verify_draft_workspace_bytes(int64_t S, int64_t D, int64_t V) {
  return verify_sizes_ok(S, D, V) ? f2i::verify_workspace_bytes(S, V) : 0;
}

int fairy2i_verify_draft(const void* p, const void* q, int p_dtype, int64_t S, int64_t D, int64_t V, const int64_t* draft,
                         const int32_t* draft_len, const float* u, const float* r, int64_t* tokens, int32_t* accepted,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!p || !draft || !u || !r || !tokens || !accepted)
    return fail(FAIRY2I_ERR_NULL, "p, draft, u, r, tokens and accepted are required");
  if (int s = check_float_dtype(p_dtype, "p_dtype")) return s;
  if (!verify_sizes_ok(S, D, V))
    return fail(FAIRY2I_ERR_SHAPE, "S = %lld, D = %lld, V = %lld: need 1 <= S <= 2^20, 1 <= D <= 63, 1 <= V <= 2^24 and "
                "S ceil(V / 4096) <= 2^23", (long long)S, (long long)D, (long long)V);
  const uint64_t e = p_dtype == FAIRY2I_BF16 ? 2 : 4;
  if (!aligned(p, e) || !aligned(q, e) || !aligned(draft, 8) || !aligned(draft_len, 4) || !aligned(u, 4) || !aligned(r, 4) ||
      !aligned(tokens, 8) || !aligned(accepted, 4))
    return fail(FAIRY2I_ERR_ALIGN, "p, q, draft, draft_len, u, r, tokens and accepted need their element's alignment");
  const uint64_t tb = (uint64_t)S * (D + 1) * 8, ab = (uint64_t)S * 4;
  const struct { const void* at; uint64_t bytes; } in[] = {
      {p, (uint64_t)S * (D + 1) * V * e}, {q, (uint64_t)S * D * V * e}, {draft, (uint64_t)S * D * 8},
      {draft_len, (uint64_t)S * 4}, {u, (uint64_t)S * D * 4}, {r, (uint64_t)S * 4}};
  for (const auto& k : in)
    if (overlap(tokens, tb, k.at, k.bytes) || overlap(accepted, ab, k.at, k.bytes))
      return fail(FAIRY2I_ERR_SHAPE, "tokens and accepted must not overlap an input");
  if (overlap(tokens, tb, accepted, ab)) return fail(FAIRY2I_ERR_SHAPE, "tokens and accepted must not overlap each other");
  if (int s = check_workspace(workspace, workspace_bytes, f2i::verify_workspace_bytes(S, V))) return s;
  const f2i::VerifyArgs a{p, q, draft, draft_len, u, r, tokens, accepted, S, V, (int)D};
  return hip_status(f2i::launch_verify(a, p_dtype == FAIRY2I_BF16, workspace, stream), "draft verification launch");
}

// ---- distillation from a teacher's top logits: the vocabulary's products with lists in place of targets ----

static constexpr int kMaxTop = 128;
static bool distill_sizes_ok(int64_t N, int64_t V, int64_t K, int64_t top) {
  return vocab_sizes_ok(N, V, K) && top >= 1 && top <= kMaxTop;
}

static int check_distill(int64_t N, int64_t V, int64_t K, int64_t top, float temperature) {
  if (int s = check_vocab_sizes(N, V, K)) return s;
  if (top < 1 || top > kMaxTop) return fail(FAIRY2I_ERR_SHAPE, "top = %lld: need 1 <= top <= %d", (long long)top, kMaxTop);
  if (!(temperature >= 0x1p-20f && temperature <= 0x1p20f))
    return fail(FAIRY2I_ERR_SHAPE, "temperature = %g: need 2^-20 to 2^20", (double)temperature);
  return FAIRY2I_OK;
}

size_t fairy2i_distill_workspace_bytes(int64_t N, int64_t V, int64_t K, int x_dtype, int top) {
  return distill_sizes_ok(N, V, K, top) ? f2i::vocab_loss_workspace_bytes(N, V, K, x_dtype == FAIRY2I_BF16, top) : 0;
}

int fairy2i_distill(const void* h, const void* W, int x_dtype, int64_t N, int64_t V, int64_t K, const int64_t* top_index,
                    const void* top_logit, int top_dtype, int top, float temperature, float* loss, float* lse,
                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!h || !W || !top_index || !top_logit || !loss || !lse)
    return fail(FAIRY2I_ERR_NULL, "h, W, top_index, top_logit, loss and lse are required");
  if (int s = check_float_dtype(x_dtype, "x_dtype")) return s;
  if (int s = check_float_dtype(top_dtype, "top_dtype")) return s;
  if (int s = check_distill(N, V, K, top, temperature)) return s;
  const uint64_t xe = x_dtype == FAIRY2I_BF16 ? 2 : 4, te = top_dtype == FAIRY2I_BF16 ? 2 : 4, ob = (uint64_t)N * 4;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(top_index, 8) || !aligned(top_logit, te) || !aligned(loss, 4) ||
      !aligned(lse, 4))
    return fail(FAIRY2I_ERR_ALIGN, "h and W need 16-byte alignment, top_index 8, top_logit its element's, loss and lse 4");
  const struct { const void* p; uint64_t bytes; } in[] = {
      {h, (uint64_t)N * K * xe}, {W, (uint64_t)V * K * xe}, {top_index, (uint64_t)N * top * 8}, {top_logit, (uint64_t)N * top * te}};
  for (const auto& r : in)
    if (overlap(loss, ob, r.p, r.bytes) || overlap(lse, ob, r.p, r.bytes))
      return fail(FAIRY2I_ERR_SHAPE, "loss and lse must not overlap h, W, top_index or top_logit");
  if (overlap(loss, ob, lse, ob)) return fail(FAIRY2I_ERR_SHAPE, "loss and lse must not overlap each other");
  if (int s = check_workspace(workspace, workspace_bytes, fairy2i_distill_workspace_bytes(N, V, K, x_dtype, top))) return s;
  f2i::VocabArgs a{};
  a.h = h; a.W = W; a.N = N; a.V = V; a.K = K; a.bf16 = x_dtype == FAIRY2I_BF16;
  a.loss = loss; a.lse_out = lse; a.ws = workspace;
  a.top_index = top_index; a.top_logit = top_logit; a.top = top; a.top_bf16 = top_dtype == FAIRY2I_BF16;
  a.temperature = temperature;
  return hip_status(f2i::launch_vocab_loss(a, stream), "distillation launch");
}

size_t fairy2i_distill_backward_workspace_bytes(int64_t N, int64_t V, int64_t K, int x_dtype, int top) {
  return distill_sizes_ok(N, V, K, top) ? f2i::vocab_loss_backward_workspace_bytes(N, V, K, x_dtype == FAIRY2I_BF16, top) : 0;
}

int fairy2i_distill_backward(const void* h, const void* W, int x_dtype, int64_t N, int64_t V, int64_t K,
                             const int64_t* top_index, const void* top_logit, int top_dtype, int top, float temperature,
                             const float* lse, const float* g, void* dh, void* dW, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
  if (!h || !W || !top_index || !top_logit || !lse || !g)
    return fail(FAIRY2I_ERR_NULL, "h, W, top_index, top_logit, lse and g are required");
  if (!dh && !dW) return fail(FAIRY2I_ERR_NULL, "one of dh and dW is required");
  if (int s = check_float_dtype(x_dtype, "x_dtype")) return s;
  if (int s = check_float_dtype(top_dtype, "top_dtype")) return s;
  if (int s = check_distill(N, V, K, top, temperature)) return s;
  const uint64_t xe = x_dtype == FAIRY2I_BF16 ? 2 : 4, te = top_dtype == FAIRY2I_BF16 ? 2 : 4;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(dh, 16) || !aligned(dW, 16) || !aligned(top_index, 8) ||
      !aligned(top_logit, te) || !aligned(lse, 4) || !aligned(g, 4))
    return fail(FAIRY2I_ERR_ALIGN, "h, W, dh and dW need 16-byte alignment, top_index 8, top_logit its element's, lse and g 4");
  const uint64_t hb = (uint64_t)N * K * xe, wb = (uint64_t)V * K * xe;
  const struct { const void* p; uint64_t bytes; } in[] = {
      {h, hb}, {W, wb}, {top_index, (uint64_t)N * top * 8}, {top_logit, (uint64_t)N * top * te}, {lse, (uint64_t)N * 4}, {g, (uint64_t)N * 4}};
  for (const auto& r : in)
    if (overlap(dh, hb, r.p, r.bytes) || overlap(dW, wb, r.p, r.bytes))
      return fail(FAIRY2I_ERR_SHAPE, "dh and dW must not overlap h, W, top_index, top_logit, lse or g");
  if (overlap(dh, hb, dW, wb)) return fail(FAIRY2I_ERR_SHAPE, "dh and dW must not overlap each other");
  if (int s = check_workspace(workspace, workspace_bytes, fairy2i_distill_backward_workspace_bytes(N, V, K, x_dtype, top)))
    return s;
  f2i::VocabArgs a{};
  a.h = h; a.W = W; a.N = N; a.V = V; a.K = K; a.bf16 = x_dtype == FAIRY2I_BF16;
  a.lse = lse; a.g = g; a.dh = dh; a.dW = dW; a.ws = workspace;
  a.top_index = top_index; a.top_logit = top_logit; a.top = top; a.top_bf16 = top_dtype == FAIRY2I_BF16;
  a.temperature = temperature;
  return hip_status(f2i::launch_vocab_loss_backward(a, stream), "distillation backward launch");
}

// Layers kept at four bits: tiles x blocks of 128 columns bounds the threads of one packing launch.
static bool w4_sizes_ok(int64_t rows, int64_t cols, int group) {
  return (group == 32 || group == 64 || group == 128) && rows >= 1 && rows <= (int64_t(1) << 24) && cols >= 1 &&
         cols <= (int64_t(1) << 20) && (rows + 15) / 16 * ((cols + 127) / 128) <= (int64_t(1) << 23);
}

static int check_w4_sizes(int64_t rows, int64_t cols, int group) {
  if (w4_sizes_ok(rows, cols, group)) return FAIRY2I_OK;
  return fail(FAIRY2I_ERR_SHAPE, "rows = %lld, cols = %lld, group = %d: need 1 <= rows <= 2^24, 1 <= cols <= 2^20, "
              "ceil(rows / 16) ceil(cols / 128) <= 2^23 and groups of 32, 64 or 128", (long long)rows, (long long)cols, group);
}

size_t fairy2i_packed_bytes_w4(int64_t rows, int64_t cols, int group, int scales_dtype) {
  if (!w4_sizes_ok(rows, cols, group) || (scales_dtype != FAIRY2I_F32 && scales_dtype != FAIRY2I_BF16)) return 0;
  return f2i::w4_bytes(rows, cols, group, scales_dtype == FAIRY2I_BF16);
}

int fairy2i_pack_w4(const uint8_t* codes, const void* scales, int scales_dtype, const uint8_t* zeros, int64_t rows,
                    int64_t cols, int group, uint8_t* packed, hipStream_t stream) {
  if (!codes || !scales || !packed) return fail(FAIRY2I_ERR_NULL, "codes, scales and packed are required");
  if (int s = check_float_dtype(scales_dtype, "scales_dtype")) return s;
  if (int s = check_w4_sizes(rows, cols, group)) return s;
  const uint64_t se = scales_dtype == FAIRY2I_BF16 ? 2 : 4, groups = (uint64_t)(cols + group - 1) / group;
  if (!aligned(packed, 16) || !aligned(scales, se))
    return fail(FAIRY2I_ERR_ALIGN, "packed needs 16-byte alignment, scales their element's");
  const uint64_t pb = f2i::w4_bytes(rows, cols, group, scales_dtype == FAIRY2I_BF16);
  if (overlap(packed, pb, codes, (uint64_t)rows * cols) || overlap(packed, pb, scales, rows * groups * se) ||
      overlap(packed, pb, zeros, rows * groups))
    return fail(FAIRY2I_ERR_SHAPE, "packed must not overlap codes, scales or zeros");
  return hip_status(f2i::launch_w4_pack(codes, scales, scales_dtype == FAIRY2I_BF16, zeros, rows, cols, group, packed, stream),
                    "four-bit pack launch");
}

int fairy2i_gemv_w4(const uint8_t* packed, int64_t rows, int64_t cols, int group, int scales_dtype, const void* x,
                    int x_dtype, int64_t B, void* y, int y_dtype, hipStream_t stream) {
  if (!packed || !x || !y) return fail(FAIRY2I_ERR_NULL, "packed, x and y are required");
  if (int s = check_float_dtype(scales_dtype, "scales_dtype")) return s;
  if (int s = check_float_dtype(x_dtype, "x_dtype")) return s;
  if (int s = check_float_dtype(y_dtype, "y_dtype")) return s;
  if (int s = check_w4_sizes(rows, cols, group)) return s;
  if (B < 1 || B > 16) return fail(FAIRY2I_ERR_SHAPE, "B = %lld: need 1 <= B <= 16", (long long)B);
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(y, 16))
    return fail(FAIRY2I_ERR_ALIGN, "packed, x and y need 16-byte alignment");
  const uint64_t yb = (uint64_t)B * rows * (y_dtype == FAIRY2I_BF16 ? 2 : 4);
  if (overlap(y, yb, packed, f2i::w4_bytes(rows, cols, group, scales_dtype == FAIRY2I_BF16)) ||
      overlap(y, yb, x, (uint64_t)B * cols * (x_dtype == FAIRY2I_BF16 ? 2 : 4)))
    return fail(FAIRY2I_ERR_SHAPE, "y must not overlap packed or x");
  const f2i::W4Args a{packed, x, y, rows, cols, group, scales_dtype == FAIRY2I_BF16, x_dtype == FAIRY2I_BF16,
                      y_dtype == FAIRY2I_BF16, (int)B};
  return hip_status(f2i::launch_w4_gemv(a, stream), "four-bit gemv launch");
}

static int64_t clip_total_pieces(int count, const int64_t* numel) {
  int64_t pieces = 0;
  for (int k = 0; k < count; ++k)
    if (numel[k] > 0) pieces += f2i::clip_pieces(numel[k]);
  return pieces;
}

size_t fairy2i_clip_grads_workspace_bytes(int count, const int64_t* numel) {
  if (count < 0 || (count > 0 && !numel)) return 0;
  return 16 + (size_t)count * sizeof(f2i::ClipItem) + (size_t)clip_total_pieces(count, numel) * sizeof(double);
}

int fairy2i_clip_grads(int count, const void* const* grads, void* const* out, const int64_t* numel, const int* dtypes,
                       float max_norm, float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (count < 0) return fail(FAIRY2I_ERR_SHAPE, "count = %d", count);
  if (!norm || (count > 0 && (!grads || !numel || !dtypes)))
    return fail(FAIRY2I_ERR_NULL, "norm and the grads, numel and dtypes arrays are required");
  if (!(max_norm >= 0.f)) return fail(FAIRY2I_ERR_SHAPE, "max_norm = %g: need max_norm >= 0", (double)max_norm);
  for (int k = 0; k < count; ++k) {
    if (numel[k] < 0 || numel[k] > (int64_t(1) << 36))
      return fail(FAIRY2I_ERR_SHAPE, "tensor %d: %lld elements out of range", k, (long long)numel[k]);
    if (int s = check_float_dtype(dtypes[k], "dtype")) return s;
    if (numel[k] == 0) continue;
    if (!grads[k] || (out && !out[k])) return fail(FAIRY2I_ERR_NULL, "tensor %d: gradient and output are required", k);
    const size_t a = dtypes[k] == FAIRY2I_BF16 ? 2 : 4;
    if (!aligned(grads[k], a) || (out && !aligned(out[k], a)))
      return fail(FAIRY2I_ERR_ALIGN, "tensor %d: gradients and outputs need their element's alignment", k);
  }
  if (!aligned(norm, 4)) return fail(FAIRY2I_ERR_ALIGN, "norm needs 4-byte alignment");
  if (int s = check_workspace(workspace, workspace_bytes, fairy2i_clip_grads_workspace_bytes(count, numel))) return s;
  {
    std::unique_ptr<Span[]> spans(new (std::nothrow) Span[2 * (size_t)count]);
    if (!spans) return fail(FAIRY2I_ERR_SHAPE, "count = %d: no host memory", count);
    int64_t n = 0;
    for (int k = 0; k < count; ++k) {
      if (numel[k] == 0) continue;
      const uint64_t bytes = (uint64_t)numel[k] * (dtypes[k] == FAIRY2I_BF16 ? 2 : 4);
      const uint64_t g = reinterpret_cast<uintptr_t>(grads[k]), o = out ? reinterpret_cast<uintptr_t>(out[k]) : g;
      spans[n++] = Span{o, o + bytes, true};
      if (o != g) spans[n++] = Span{g, g + bytes, false};
    }
    if (written_twice(spans.get(), n))
      return fail(FAIRY2I_ERR_SHAPE, "a tensor is listed twice, or an output overlaps another output or a gradient");
    // the norm is stored before the gradients are read for the second time
    const uint64_t at = reinterpret_cast<uintptr_t>(norm);
    for (int64_t k = 0; k < n; ++k) {
      if (at >= spans[k].hi || at + 4 <= spans[k].lo) continue;
      int dev = 0;                                   // without a device every call returns FAIRY2I_ERR_HIP
      if (const hipError_t e = hipGetDevice(&dev); e != hipSuccess) return hip_status(e, "hipGetDevice");
      return fail(FAIRY2I_ERR_SHAPE, "norm overlaps a gradient or an output");
    }
  }
  // workspace: coefficient, table (8-byte entries), partial sums
  float* coef = static_cast<float*>(workspace);
  f2i::ClipItem* table = reinterpret_cast<f2i::ClipItem*>(static_cast<uint8_t*>(workspace) + 16);
  double* part = reinterpret_cast<double*>(table + count);
  int64_t pieces = 0;
  int items = 0;
  hipError_t e = hipSuccess;
  for (int k = 0; k < count;) {
    f2i::ClipGroup grp;
    grp.count = 0;
    for (; k < count && grp.count < f2i::kMaxClipItems; ++k) {
      if (numel[k] == 0) continue;
      void* o = out ? out[k] : const_cast<void*>(grads[k]);
      const int flags = (dtypes[k] == FAIRY2I_BF16 ? f2i::kClipBf16 : 0) |
                        (aligned(grads[k], 16) && aligned(o, 16) ? f2i::kClipVec : 0);
      grp.items[grp.count++] = f2i::ClipItem{grads[k], o, pieces, (uint16_t)f2i::clip_tail(numel[k]), (uint16_t)flags};
      pieces += f2i::clip_pieces(numel[k]);
    }
    if (grp.count == 0) continue;
    e = f2i::launch_clip_table(grp, table + items, stream);
    if (e != hipSuccess) return hip_status(e, "gradient clipping launch");
    items += grp.count;
  }
  e = f2i::launch_clip_square(table, items, pieces, part, stream);
  if (e != hipSuccess) return hip_status(e, "gradient norm launch");
  e = f2i::launch_clip_norm(part, pieces, max_norm, norm, coef, stream);
  if (e != hipSuccess) return hip_status(e, "gradient norm launch");
  e = f2i::launch_clip_scale(table, items, pieces, coef, stream);
  if (e != hipSuccess) return hip_status(e, "gradient clipping launch");
  return ok();
}

}  // extern "C"
