// Verification of drafted tokens: with target probabilities p and draft probabilities q, token x_j is kept
// while u_j q_j(x_j) < p_j(x_j); the next token is drawn from w = max(p_a - q_a, 0) at the first refused
// position a (from p_a where that leaves nothing), or from p behind the last draft: the lowest v with
// sum_{v' <= v} w_v' > r sum w.
//
// Products and differences of fp32 or bf16 values are exact in fp64 (up to the last bits of a difference),
// and the sums are fp64, so that a token depends on their order only where r falls within 1e-15 of a border.
// Two launches: every workgroup finds its sequence's position again and sums one piece of its rows of p and
// q; then one workgroup a sequence finds the piece in which r falls and reads it a second time.
#include "common.hpp"

namespace f2i {

namespace {

constexpr int kPiece = 4096;             // entries of a row per workgroup
constexpr int kThreads = 256;
constexpr int kEach = kPiece / kThreads;

__device__ __forceinline__ float entry(const float* p, int64_t at) { return p[at]; }
__device__ __forceinline__ float entry(const uint16_t* p, int64_t at) { return __uint_as_float((uint32_t)p[at] << 16); }

// Where a sequence's drafts end: the number kept, and whether one was refused there.
struct Stop {
  int kept;
  bool refused;
};

// Each wave by itself, one draft a lane.
template <typename T>
__device__ __forceinline__ Stop find_stop(const VerifyArgs& a, int64_t s) {
  const int lane = threadIdx.x & (kWave - 1);
  const int len = a.draft_len ? min(max(a.draft_len[s], 0), a.D) : a.D;
  bool keep = false;
  if (lane < len) {
    const int64_t x = a.draft[s * a.D + lane];
    if (x >= 0 && x < a.V) {
      const double p = entry(static_cast<const T*>(a.p), (s * (a.D + 1) + lane) * a.V + x);
      const double q = a.q ? (double)entry(static_cast<const T*>(a.q), (s * a.D + lane) * a.V + x) : 1.0;
      keep = (double)a.u[s * a.D + lane] * q < p;
    }
  }
  const uint64_t out = ~__ballot(keep);
  const int kept = out ? __builtin_ctzll(out) : kWave;
  return Stop{__builtin_amdgcn_readfirstlane(kept), kept < len};
}

// The weights of a row's entries: (difference, p itself), 0 for values that are not positive or not finite.
template <typename T>
struct Row {
  const T* p;
  const T* q;          // null: a greedy draft, whose whole probability lies at x
  int64_t x;
  bool refused;
  __device__ Row(const VerifyArgs& a, int64_t s, const Stop& stop)
      : p(static_cast<const T*>(a.p) + (s * (a.D + 1) + stop.kept) * a.V),
        q(a.q && stop.refused ? static_cast<const T*>(a.q) + (s * a.D + stop.kept) * a.V : nullptr),
        x(stop.refused ? a.draft[s * a.D + stop.kept] : -1), refused(stop.refused) {}
  __device__ __forceinline__ static double positive(double w) { return w > 0.0 && w < INFINITY ? w : 0.0; }
  __device__ __forceinline__ double2 weights(int64_t v) const {
    const double pv = entry(p, v);
    const double rest = q ? pv - (double)entry(q, v) : v == x ? 0.0 : pv;
    return make_double2(refused ? positive(rest) : 0.0, positive(pv));
  }
};

__device__ __forceinline__ double wave_scan(double v) {      // inclusive
  const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const double o = __shfl_up(v, off);
    if (lane >= off) v += o;
  }
  return v;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_verify_sums(VerifyArgs a, int pieces, double2* __restrict__ sums) {
  __shared__ double2 s_sum[kThreads / kWave];
  const int64_t s = blockIdx.x / pieces;
  const int piece = blockIdx.x - (int)(s * pieces);
  const Row<T> row(a, s, find_stop<T>(a, s));
  double2 sum = make_double2(0.0, 0.0);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int64_t v = (int64_t)piece * kPiece + k * kThreads + threadIdx.x;
    if (v >= a.V) continue;
    const double2 w = row.weights(v);
    sum.x += w.x;
    sum.y += w.y;
  }
  sum.x = wave_sum(sum.x);
  sum.y = wave_sum(sum.y);
  if ((threadIdx.x & (kWave - 1)) == 0) s_sum[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / kWave; ++w) {
      sum.x += s_sum[w].x;
      sum.y += s_sum[w].y;
    }
    sums[blockIdx.x] = sum;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_verify_pick(VerifyArgs a, int pieces, const double2* __restrict__ sums) {
  __shared__ double s_wave[kThreads / kWave];
  __shared__ int s_found[kThreads / kWave], s_last[kThreads / kWave];
  const int64_t s = blockIdx.x;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const Stop stop = find_stop<T>(a, s);
  const Row<T> row(a, s, stop);
  const double2* __restrict__ mine = sums + s * pieces;
  // every wave finds the piece for itself: the total first, then the first piece past r of it
  double2 total = make_double2(0.0, 0.0);
  for (int k = 0; k < pieces; k += kWave) {
    const double2 w = k + lane < pieces ? mine[k + lane] : make_double2(0.0, 0.0);
    total.x += __shfl(wave_scan(w.x), kWave - 1);
    total.y += __shfl(wave_scan(w.y), kWave - 1);
  }
  const bool rest = total.x > 0.0;
  const double all = rest ? total.x : total.y;
  const double goal = (double)a.r[s] * all;
  int piece = -1, last = -1;                                  // last: the last piece with any weight
  double before = 0.0, before_last = 0.0, carry = 0.0;
  for (int k = 0; k < pieces && piece < 0; k += kWave) {
    const double2 w = k + lane < pieces ? mine[k + lane] : make_double2(0.0, 0.0);
    const double v = rest ? w.x : w.y, upto = carry + wave_scan(v);
    if (const uint64_t over = __ballot(v > 0.0 && upto > goal)) {
      const int at = __builtin_ctzll(over);
      piece = k + at;
      before = __shfl(upto - v, at);
    }
    if (const uint64_t some = __ballot(v > 0.0)) {
      const int at = kWave - 1 - __builtin_clzll(some);
      last = k + at;
      before_last = __shfl(upto - v, at);
    }
    carry = __shfl(upto, kWave - 1);
  }
  if (piece < 0) {
    piece = last;
    before = before_last;
  }
  int token = -1;                                             // no weight at all
  if (piece >= 0) {
    double w[kEach], sum = 0.0;
    const int64_t v0 = (int64_t)piece * kPiece + threadIdx.x * kEach;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      w[k] = 0.0;
      if (v0 + k < a.V) {
        const double2 both = row.weights(v0 + k);
        w[k] = rest ? both.x : both.y;
      }
      sum += w[k];
    }
    const double upto = wave_scan(sum);
    if (lane == kWave - 1) s_wave[wave] = upto;
    __syncthreads();
    double run = before + (upto - sum);
    for (int k = 0; k < wave; ++k) run += s_wave[k];
    int found = kPiece, end = -1;                             // within the piece; entries with weight only
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      run += w[k];
      if (w[k] > 0.0) {
        end = threadIdx.x * kEach + k;
        if (run > goal) found = min(found, end);
      }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      found = min(found, __shfl_xor(found, off));
      end = max(end, __shfl_xor(end, off));
    }
    if (lane == 0) {
      s_found[wave] = found;
      s_last[wave] = end;
    }
    __syncthreads();
    for (int k = 0; k < kThreads / kWave; ++k) {
      found = min(found, s_found[k]);
      end = max(end, s_last[k]);
    }
    token = piece * kPiece + (found < kPiece ? found : end);
  }
  if (threadIdx.x <= a.D) {
    const int j = threadIdx.x;
    a.tokens[s * (a.D + 1) + j] = j < stop.kept ? a.draft[s * a.D + j] : j == stop.kept ? token : -1;
  }
  if (threadIdx.x == 0) a.accepted[s] = stop.kept;
}

template <typename T>
hipError_t verify_t(const VerifyArgs& a, void* ws, hipStream_t s) {
  const int pieces = (int)((a.V + kPiece - 1) / kPiece);
  double2* sums = static_cast<double2*>(ws);
  hipLaunchKernelGGL((k_verify_sums<T>), dim3((unsigned)(a.S * pieces)), dim3(kThreads), 0, s, a, pieces, sums);
  hipLaunchKernelGGL((k_verify_pick<T>), dim3((unsigned)a.S), dim3(kThreads), 0, s, a, pieces, sums);
  return hipGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int64_t S, int64_t V) { return (size_t)S * ((V + kPiece - 1) / kPiece) * sizeof(double2); }

hipError_t launch_verify(const VerifyArgs& a, int bf16, void* ws, hipStream_t s) {
  return bf16 ? verify_t<uint16_t>(a, ws, s) : verify_t<float>(a, ws, s);
}

}  // namespace f2i
