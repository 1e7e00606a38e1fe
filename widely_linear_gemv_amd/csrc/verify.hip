// Verification of drafted tokens: with target probabilities p and draft probabilities q, token x_j is kept
// while u_j q_j(x_j) < p_j(x_j); the next token is drawn from w = max(p_a - q_a, 0) at the first refused
// position a (from p_a where that leaves nothing), or from p behind the last draft: the lowest v with
// sum_{v' <= v} w_v' > r sum w.
//
// Products and differences of fp32 or bf16 values are exact in fp64 (up to the last bits of a difference),
// and the sums are fp64, so that a token depends on their order only where r falls within 1e-15 of a border.
// A wave sums a contiguous piece of the rows of p and q; the piece in which r falls is then read a second time
// by one wave.  Where a sequence has a workgroup to itself that is one launch; where there are few sequences and
// a large vocabulary a first launch spreads the sums over the device.  Which entries have weight is decided in
// fp32 (a difference's sign is exact there): 9 instructions an entry instead of 16 count where one CU does all.
#include "tiles.hpp"

namespace f2i {

namespace {

constexpr int kWaves = 16;               // of a sequence's workgroup (one launch)
constexpr int kPiece = 2048;             // entries of a wave's piece (two launches)
constexpr int kPieceWaves = 4;

__device__ __forceinline__ float entry(const float* p, int64_t at) { return p[at]; }
__device__ __forceinline__ float entry(const uint16_t* p, int64_t at) { return __uint_as_float((uint32_t)p[at] << 16); }

// 16 bytes of a row, at any element's alignment.
template <typename T>
struct Entries {
  static constexpr int kCount = 16 / sizeof(T);
  struct __attribute__((packed, aligned(sizeof(T)))) Raw { v4u v; } raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const Raw*>(p); }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(raw.v[e]);
    else return e & 1 ? bf16_hi(raw.v[e / 2]) : bf16_lo(raw.v[e / 2]);
  }
};

// Where a sequence's drafts end: the number kept, and whether one was refused there (then the draft's token).
struct Stop {
  int kept;
  bool refused;
  int64_t x;
};

// Each wave by itself, one draft a lane.
template <typename T>
__device__ __forceinline__ Stop find_stop(const VerifyArgs& a, int64_t s) {
  const int lane = threadIdx.x & (kWave - 1);
  // all loads that depend on nothing first
  const int len = a.draft_len ? min(max(a.draft_len[s], 0), a.D) : a.D;
  const int64_t x = lane < a.D ? a.draft[s * a.D + lane] : -1;
  const float u = lane < a.D ? a.u[s * a.D + lane] : 0.f;
  bool keep = false;
  if (lane < len && x >= 0 && x < a.V) {
    const double p = entry(static_cast<const T*>(a.p), (s * (a.D + 1) + lane) * a.V + x);
    const double q = a.q ? (double)entry(static_cast<const T*>(a.q), (s * a.D + lane) * a.V + x) : 1.0;
    keep = (double)u * q < p;
  }
  const int kept = __builtin_ctzll(~__ballot(keep));          // lane 63 has no draft
  return Stop{__builtin_amdgcn_readfirstlane(kept), kept < len, kept < len ? __shfl(x, kept) : -1};
}

// The weights of a row's entries: p, or p - q (PAIR), where that is positive and in fp32's range, and 0 elsewhere.
// (A load that depended on a condition would make the compiler wait for each one: hence the types.)
template <typename T, bool PAIR>
struct Row {
  using E = Entries<T>;
  static constexpr int kStep = E::kCount * kWave;      // entries of a wave's load
  static constexpr int kBatch = 2048 / kStep;          // loads of a row in flight
  const T* p;
  const T* q;
  int V, x;            // x: an entry without weight (a greedy draft's token), or -1
  __device__ __forceinline__ double weigh(float pv, float qv, int v) const {
    const float d = PAIR ? pv - qv : pv;
    const bool has = __float_as_uint(d) - 1u < 0x7F7FFFFFu && (PAIR || v != x);      // 0 < d < infinity
    return has ? (PAIR ? (double)pv - (double)qv : (double)pv) : 0.0;
  }
  // f(e, weight) of a lane's entries in the step at v0, which lies inside the row
  struct Raw {
    E p, q;
  };
  __device__ __forceinline__ Raw load(int v0) const {
    const int v = v0 + (threadIdx.x & (kWave - 1)) * E::kCount;
    Raw r;
    r.p.load(p + v);
    if constexpr (PAIR) r.q.load(q + v);
    return r;
  }
  template <typename F>
  __device__ __forceinline__ void each(const Raw& r, int v0, F f) const {
    const int v = v0 + (threadIdx.x & (kWave - 1)) * E::kCount;
#pragma unroll
    for (int e = 0; e < E::kCount; ++e) f(e, weigh(r.p[e], PAIR ? r.q[e] : 0.f, v + e));
  }
  // the same in a step that the row may end in
  template <typename F>
  __device__ __forceinline__ void each_end(int v0, F f) const {
    const int v = v0 + (threadIdx.x & (kWave - 1)) * E::kCount;
#pragma unroll
    for (int e = 0; e < E::kCount; ++e)
      f(e, v + e < V ? weigh(entry(p, v + e), PAIR ? entry(q, v + e) : 0.f, v + e) : 0.0);
  }
  // the sum of the entries from v0 on, up to v1 or the row's end, in every lane
  __device__ __forceinline__ double sum(int v0, int v1) const {
    double sum = 0.0;
    v1 = min(v1, V);
    const auto add = [&](int, double w) { sum += w; };
    int v = v0;
    for (; v + kBatch * kStep <= v1; v += kBatch * kStep) {
      Raw r[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) r[k] = load(v + k * kStep);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) each(r[k], v + k * kStep, add);
    }
    for (; v + kStep <= v1; v += kStep) each(load(v), v, add);
    if (v < v1) each_end(v, add);
    return wave_sum(sum);
  }
  // the first entry with weight, from v0 on, at which `before` and the weights up to it pass `goal`, or the last
  // with weight; -1 if none has any
  __device__ __forceinline__ int find(int v0, int v1, double before, double goal) const;
};

// f(row) for the weights that a sequence's next token is drawn from: what the target has above the draft, or (all)
// the target's own.
template <typename T, typename F>
__device__ __forceinline__ void with_row(const VerifyArgs& a, int64_t s, const Stop& stop, bool all, F f) {
  const T* p = static_cast<const T*>(a.p) + (s * (a.D + 1) + stop.kept) * a.V;
  if (a.q && !all) f(Row<T, true>{p, static_cast<const T*>(a.q) + (s * a.D + stop.kept) * a.V, (int)a.V, -1});
  else f(Row<T, false>{p, nullptr, (int)a.V, all || stop.x < 0 || stop.x >= a.V ? -1 : (int)stop.x});
}

__device__ __forceinline__ double wave_scan(double v) {      // inclusive
  const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const double o = __shfl_up(v, off);
    if (lane >= off) v += o;
  }
  return v;
}

template <typename T, bool PAIR>
__device__ __forceinline__ int Row<T, PAIR>::find(int v0, int v1, double before, double goal) const {
  v1 = min(v1, V);
  // the step in which it lies
  int last = -1;
  double before_last = before;
  bool found = false;
  const auto look = [&](int at, double sum) {
    if (!found && sum > 0.0) {
      last = at;
      before_last = before;
      found = before + sum > goal;
    }
    before += sum;
  };
  int v = v0;
  for (; v + kBatch * kStep <= v1 && !found; v += kBatch * kStep) {
    Raw r[kBatch];
    double sum[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) r[k] = load(v + k * kStep);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      sum[k] = 0.0;
      each(r[k], v + k * kStep, [&](int, double w) { sum[k] += w; });
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) sum[k] = wave_sum(sum[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) look(v + k * kStep, sum[k]);
  }
  for (; v < v1 && !found; v += kStep) {
    double sum = 0.0;
    each_end(v, [&](int, double w) { sum += w; });
    look(v, wave_sum(sum));
  }
  if (last < 0) return -1;
  // the entry: with weight, the first past the goal or the step's last
  double w[E::kCount], sum = 0.0;
  each_end(last, [&](int e, double weight) {
    w[e] = weight;
    sum += weight;
  });
  double run = before_last + (wave_scan(sum) - sum);
  int over = -1, end = -1;
#pragma unroll
  for (int e = 0; e < E::kCount; ++e) {
    run += w[e];
    if (w[e] > 0.0) {
      end = e;
      if (over < 0 && run > goal) over = e;
    }
  }
  const uint64_t past = __ballot(over >= 0), some = __ballot(end >= 0);
  const int l = past ? __builtin_ctzll(past) : kWave - 1 - __builtin_clzll(some);
  return last + l * E::kCount + __shfl(past ? over : end, l);
}

// Where the next token lies, from the sums of a row's pieces in order (sign -1: from those that are under 0, as if
// they were above): in every lane of a wave.
struct Spot {
  int piece;            // -1: no weight at all
  double before, goal;  // weights before the piece, r times all
};
__device__ __forceinline__ Spot find_spot(const double* sums, int pieces, double r, double sign = 1.0) {
  const int lane = threadIdx.x & (kWave - 1);
  const auto load = [&](int k) { return k + lane < pieces ? fmax(sign * sums[k + lane], 0.0) : 0.0; };
  double total = 0.0;
  for (int k = 0; k < pieces; k += kWave) total += wave_sum(load(k));
  Spot last{-1, 0.0, r * total};                              // the last piece with any weight
  double carry = 0.0;
  for (int k = 0; k < pieces; k += kWave) {
    const double v = load(k), upto = carry + wave_scan(v);
    const uint64_t over = __ballot(v > 0.0 && upto > last.goal), some = __ballot(v > 0.0);
    if (some) {
      const int at = over ? __builtin_ctzll(over) : kWave - 1 - __builtin_clzll(some);
      last.piece = k + at;
      last.before = __shfl(upto - v, at);
      if (over) break;
    }
    carry = __shfl(upto, kWave - 1);
  }
  return last;
}

// One wave: the outputs of sequence s.
__device__ __forceinline__ void store(const VerifyArgs& a, int64_t s, const Stop& stop, int64_t token) {
  const int lane = threadIdx.x & (kWave - 1);
  if (lane <= a.D)
    a.tokens[s * (a.D + 1) + lane] = lane < stop.kept ? a.draft[s * a.D + lane] : lane == stop.kept ? token : -1;
  if (lane == 0) a.accepted[s] = stop.kept;
}

// One launch: a workgroup a sequence.
template <typename T>
__global__ __launch_bounds__(kWaves* kWave) void k_verify(VerifyArgs a, int each) {
  __shared__ double s_sums[kWaves];
  const int64_t s = blockIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const Stop stop = find_stop<T>(a, s);
  const double r = a.r[s];
  // the rest of the target's probability; if that leaves nothing, all of it
  for (bool all = !stop.refused;; all = true) {
    double sum;
    with_row<T>(a, s, stop, all, [&](const auto& row) { sum = row.sum(wave * each, (wave + 1) * each); });
    if ((threadIdx.x & (kWave - 1)) == 0) s_sums[wave] = sum;
    __syncthreads();
    const Spot spot = find_spot(s_sums, kWaves, r);
    if (spot.piece < 0 && !all) {
      __syncthreads();
      continue;
    }
    if (wave != 0) return;
    int token = -1;
    if (spot.piece >= 0)
      with_row<T>(a, s, stop, all, [&](const auto& row) {
        token = row.find(spot.piece * each, (spot.piece + 1) * each, spot.before, spot.goal);
      });
    return store(a, s, stop, token);
  }
}

// Two launches: every wave finds its sequence's position again and sums a piece; then a wave a sequence, which
// finds the position behind the sums.  A piece in which the draft leaves nothing of the target gives the target's
// own sum instead, under 0: if that is so in every piece, the token is drawn from those, and still from one piece
// that is read a second time.  (That wave summing the whole row by itself: 64 refused sequences of 131072 147 us, one
// of 2^24 9.2 ms; so 22 us and 0.2 ms.)
template <typename T>
__global__ __launch_bounds__(kPieceWaves* kWave) void k_verify_sums(VerifyArgs a, int groups, int pieces,
                                                                     double* __restrict__ sums) {
  const int64_t s = blockIdx.x / groups;
  const int piece = (blockIdx.x - (int)(s * groups)) * kPieceWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (piece >= pieces) return;
  const Stop stop = find_stop<T>(a, s);
  double sum;
  with_row<T>(a, s, stop, !stop.refused, [&](const auto& row) { sum = row.sum(piece * kPiece, (piece + 1) * kPiece); });
  if (stop.refused && sum == 0.0)
    with_row<T>(a, s, stop, true, [&](const auto& row) { sum = -row.sum(piece * kPiece, (piece + 1) * kPiece); });
  if (threadIdx.x & (kWave - 1)) return;
  sums += s * (pieces + 2);
  sums[piece] = sum;
  if (piece == 0) {
    sums[pieces] = stop.kept;
    sums[pieces + 1] = stop.refused;
  }
}

template <typename T>
__global__ __launch_bounds__(kWave) void k_verify_pick(VerifyArgs a, int pieces, const double* __restrict__ sums) {
  const int64_t s = blockIdx.x;
  sums += s * (pieces + 2);
  const int kept = __builtin_amdgcn_readfirstlane((int)sums[pieces]);
  const bool refused = sums[pieces + 1] != 0.0;
  const Stop stop{kept, refused, refused ? a.draft[s * a.D + kept] : -1};
  const double r = a.r[s];
  Spot spot = find_spot(sums, pieces, r);
  const bool all = !refused || spot.piece < 0;
  if (refused && all) spot = find_spot(sums, pieces, r, -1.0);
  int token = -1;
  if (spot.piece >= 0)
    with_row<T>(a, s, stop, all, [&](const auto& row) {
      token = row.find(spot.piece * kPiece, (spot.piece + 1) * kPiece, spot.before, spot.goal);
    });
  store(a, s, stop, token);
}

int pieces_of(int64_t V) { return (int)((V + kPiece - 1) / kPiece); }

// One workgroup a sequence, or two launches.  fp32 p and q, kernels in a row, one launch and two: one sequence of
// 5003 entries 5.7 and 8.2 us, 32000 8.0 and 8.4, 40960 8.6 and 8.7, 50257 12.9 and 8.6, 131072 16.9 and 8.6; 64
// sequences 6.8 and 10.3, 8.6 and 9.3, 10.6 and 10.0, 14.1 and 10.7, 24.0 and 17.1; 256, one a CU, 7.1 and 10.3, 15.4
// and 18.3, 17.3 and 18.5, 22.7 and 22.0, 45.1 and 40.1; 512, two a CU, 12.6 and 11.4, 28.7 and 27.3, 31.1 and 28.4.
// (bf16, 256: 7.9 and 11.0, 11.1 and 14.5, 11.6 and 14.1, 17.8 and 18.3; 512: 14.2 and 11.9, 24.1 and 22.6.)
bool alone(int64_t S, int64_t V) { return V <= 40960 && S <= 256; }

template <typename T>
hipError_t verify_t(const VerifyArgs& a, void* ws, hipStream_t s) {
  if (alone(a.S, a.V)) {
    const int step = Row<T, true>::kStep, each = (int)((a.V + kWaves * step - 1) / (kWaves * step)) * step;
    hipLaunchKernelGGL((k_verify<T>), dim3((unsigned)a.S), dim3(kWaves * kWave), 0, s, a, each);
    return hipGetLastError();
  }
  const int pieces = pieces_of(a.V), groups = (pieces + kPieceWaves - 1) / kPieceWaves;
  double* sums = static_cast<double*>(ws);
  hipLaunchKernelGGL((k_verify_sums<T>), dim3((unsigned)(a.S * groups)), dim3(kPieceWaves * kWave), 0, s, a, groups, pieces,
                     sums);
  hipLaunchKernelGGL((k_verify_pick<T>), dim3((unsigned)a.S), dim3(kWave), 0, s, a, pieces, sums);
  return hipGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int64_t S, int64_t V) { return alone(S, V) ? 0 : (size_t)S * (pieces_of(V) + 2) * sizeof(double); }

hipError_t launch_verify(const VerifyArgs& a, int bf16, void* ws, hipStream_t s) {
  return bf16 ? verify_t<uint16_t>(a, ws, s) : verify_t<float>(a, ws, s);
}

}  // namespace f2i
