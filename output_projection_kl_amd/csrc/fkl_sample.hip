// Sampling on gfx950 (fkl_sample): one entry of each row of logits, with
// temperature, top-k, top-p and min-p, from a given random number.
//
// What is kept of a row is a prefix of its entries ordered by (logit
// descending, position ascending), so it is held as a border: every entry
// above the border's logit, and those equal to it up to a position. The draw
// runs over the kept entries in the order of positions.
//
// Whether a token is drawn goes by sums over up to V weights, compared with
// each other: the weights exp((x - m) / T) and their sums are in fp64, where
// two orders of summation differ by less than 1e-15 of the total, far below
// the smallest weight that is ever drawn in practice.
//
// Three routes, by the row length:
//   up to 1024 entries: k_sample_short, one wave per row, the row in registers.
//   up to 2^18: k_sample_scan reads the logits once, spread over all CUs, and
//     leaves per row the largest logit of every 64 entries and, where the
//     filters need it, the mass or a mass histogram of every chunk;
//     k_sample_pick, one workgroup per row, bounds the border from those,
//     reads again only the groups that reach the bound (or one chunk), and
//     settles the border and the draw exactly among them.
//   longer rows, and rows whose border the bound leaves too wide (thousands of
//     equal logits, thousands of entries kept by top-k): sample_row_exact, one
//     workgroup per row, radix selection over the row itself.
#include <algorithm>

#include "fkl_decode.h"
#include "fkl_device.h"

namespace fkl {

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;
constexpr uint32_t kMaskedKey = 0x007fffffu;  // the key of -inf

// Order-preserving bits of a logit: NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t logit_key(float v) {
  v = v != v ? -INFINITY : v + 0.0f;
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// 2^t in fp64 for t <= 0: t = n + f with |f| <= 1/2, the Taylor series of
// exp(f ln 2) to the 12th power (remainder below 0.3466^13 / 13! = 1.7e-16).
// Below the smallest normal number the result is 0.
__device__ __forceinline__ double exp2_neg(double t) {
  if (!(t > -1022.0)) return 0.0;
  const double n = rint(t);
  const double y = (t - n) * 0.69314718055994530942;
  double s = 1.0 / 479001600.0;
  s = fma(s, y, 1.0 / 39916800.0);
  s = fma(s, y, 1.0 / 3628800.0);
  s = fma(s, y, 1.0 / 362880.0);
  s = fma(s, y, 1.0 / 40320.0);
  s = fma(s, y, 1.0 / 5040.0);
  s = fma(s, y, 1.0 / 720.0);
  s = fma(s, y, 1.0 / 120.0);
  s = fma(s, y, 1.0 / 24.0);
  s = fma(s, y, 1.0 / 6.0);
  s = fma(s, y, 0.5);
  s = fma(s, y, 1.0);
  s = fma(s, y, 1.0);
  return ldexp(s, static_cast<int>(n));
}

// Geometry of the scan. A row is read in 16-byte pieces at 16-byte aligned
// addresses: element e of the row's pieces is position e - lead, lead the
// elements between the aligned address and the row's start.
constexpr int kGroup = 64;                 // elements per recorded maximum
constexpr int kScanElems = 16;             // elements per thread of a scan workgroup
constexpr int kScanBins = 512;             // mass histogram: bins of 1/16 bit below the chunk's maximum
constexpr int kCandidates = 4096;          // entries that k_sample_pick settles in LDS
constexpr int kShortRow = 1024;

struct SampleParams {
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  int64_t ld_ids;
  const float* u;
  fkl_sample_params set;
  int32_t* token;
  float* logprob;
  int32_t V;
  int64_t row0;    // first row of this launch
  // k_sample_scan's results, per row: the maximum of each group, and per
  // chunk of chunk_elems elements its maximum, mass and mass histogram
  uint32_t* group_max;
  uint32_t* chunk_max;
  double* chunk_mass;
  uint64_t* chunk_hist;
  int32_t groups, chunks, chunk_elems;
  DebugCheck dbg;  // debug build: span 0 = logits, 1 = ids, 2 = u, 3 = token, 4 = logprob
};

// One row's settings in the form that the kernels use.
struct RowSettings {
  bool valid;
  double c;     // log2(e) / T
  uint32_t k;   // entries kept at most; V when off
  double p;     // >= 1 when off
  double q;     // <= 0 when off
  double u;
};

__device__ __forceinline__ RowSettings row_settings(const SampleParams& P, int64_t row) {
  const float T = P.set.temperature_rows ? P.set.temperature_rows[row] : P.set.temperature;
  const int32_t k = P.set.top_k_rows ? P.set.top_k_rows[row] : P.set.top_k;
  const float p = P.set.top_p_rows ? P.set.top_p_rows[row] : P.set.top_p;
  const float q = P.set.min_p_rows ? P.set.min_p_rows[row] : P.set.min_p;
  const float u = dload(P.dbg, 2, kDbgSampleLogits, P.u + row);
  RowSettings s;
  s.valid = T >= 0.0f && T < INFINITY;
  // the first entry alone: greedy, or a filter that only it can pass
  const bool first = T == 0.0f || p <= 0.0f || q > 1.0f;
  s.k = first ? 1u : (k <= 0 || k > P.V) ? static_cast<uint32_t>(P.V) : static_cast<uint32_t>(k);
  s.c = T > 0.0f ? 1.4426950408889634074 / static_cast<double>(T) : 1.0;
  s.p = first || !(p < 1.0f) ? 1.0 : static_cast<double>(p);
  s.q = first || !(q > 0.0f) ? 0.0 : static_cast<double>(q);
  s.u = u > 0.0f ? static_cast<double>(fminf(u, 1.0f)) : 0.0;
  return s;
}

// What the scan leaves for a row beside the maxima: nothing where top-k or
// min-p bound the border by themselves, each chunk's mass where the whole
// row's mass counts, each chunk's mass histogram where top-p alone decides.
enum RowMode { kMaximaOnly, kChunkMass, kMassHistogram };

__device__ __forceinline__ RowMode row_mode(const RowSettings& s, int V) {
  if (s.k < static_cast<uint32_t>(V)) return kMaximaOnly;
  if (s.p < 1.0) return s.q > 0.0 ? kChunkMass : kMassHistogram;
  return s.q > 0.0 ? kMaximaOnly : kChunkMass;
}

// Weight of an entry relative to the row's largest logit m.
__device__ __forceinline__ double weight_of(uint32_t key, float m, uint32_t m_key, double c) {
  if (key == m_key) return 1.0;
  if (key <= kMaskedKey) return 0.0;
  return exp2_neg((static_cast<double>(key_logit(key)) - static_cast<double>(m)) * c);
}

__device__ __forceinline__ double shfl_xor_f64(double v, int mask) { return __shfl_xor(v, mask, 64); }

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += shfl_xor_f64(v, o);
  return v;
}

// The first position of [0, V) at which the running sum of weight(position)
// exceeds target (the last position of positive weight if rounding leaves
// none; -1 if no weight is positive). Halves the row sixteen ways at a time:
// each wave sums one part, the part holding the target is divided again, and
// the last 1024 positions or fewer are scanned 64 to a wave. Every thread
// returns the same.
template <class Weight>
__device__ int find_position(Weight weight, int V, double target, double* shared) {
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  int lo = 0, n = V;
  double base = 0.0;
  for (;;) {
    const bool leaf = n <= kRowThreads;
    const int part = leaf ? 64 : (n + kRowWaves * 64 - 1) / (kRowWaves * 64) * 64;
    const int b = min(lo + wave * part, lo + n);
    const int e = min(b + part, lo + n);
    double s = 0.0;
    for (int i = b + lane; i < e; i += 64) s += weight(i);
    const double mine = s;
    s = wave_sum_f64(s);
    __syncthreads();
    if (lane == 0) shared[wave] = s;
    __syncthreads();
    int at = -1;
    double at_base = base, run = base;
    bool found = false;
    for (int w = 0; w < kRowWaves; ++w) {
      const double t = shared[w];
      if (!found && t > 0.0) {
        at = w;
        at_base = run;
        found = run + t > target;
      }
      run += t;
    }
    if (at < 0) return -1;
    if (!leaf) {
      const int nlo = lo + at * part;
      n = min(part, lo + n - nlo);
      lo = nlo;
      base = at_base;
      continue;
    }
    if (wave == at) {
      double incl = mine;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(incl, o, 64);
        if (lane >= o) incl += y;
      }
      const uint64_t hit = __ballot(mine > 0.0 && at_base + incl > target);
      const uint64_t any = __ballot(mine > 0.0);
      const int l = hit ? __ffsll(static_cast<long long>(hit)) - 1 : 63 - __clzll(static_cast<long long>(any));
      if (lane == 0) shared[kRowWaves] = static_cast<double>(b + l);
    }
    __syncthreads();
    const int pos = static_cast<int>(shared[kRowWaves]);
    __syncthreads();
    return pos;
  }
}

// Sum over the block of each thread's v, in a fixed order.
__device__ __forceinline__ double block_sum_f64(double v, double* shared) {
  v = wave_sum_f64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kRowWaves; ++w) s += shared[w];
  return s;
}

__device__ __forceinline__ void put_none(const SampleParams& P, int64_t row) {
  dstore(P.dbg, 3, kDbgSampleOut, P.token + row, int32_t(-1));
  if (P.logprob) dstore(P.dbg, 4, kDbgSampleOut, P.logprob + row, -INFINITY);
}

__device__ __forceinline__ void put_draw(const SampleParams& P, int64_t row, int at, double prob) {
  const int32_t id = P.ids ? dload(P.dbg, 1, kDbgSampleLogits, P.ids + row * P.ld_ids + at) : at;
  dstore(P.dbg, 3, kDbgSampleOut, P.token + row, id);
  if (P.logprob) dstore(P.dbg, 4, kDbgSampleOut, P.logprob + row, static_cast<float>(log(prob)));
}

constexpr int kDigits = 256;

// Shared memory of sample_row_exact.
struct ExactLds {
  double part[kRowWaves + 1];
  uint64_t mass[kDigits];
  uint32_t count[kDigits];
  uint32_t pick[2];
  uint64_t pick_mass[2];
};

// One workgroup, any row: the border by radix selection over the row's
// keys, eight bits at a time, first by count (top-k), then by mass (top-p),
// and the draw by find_position. The masses of the selection are integers in
// units of 2^-shift, whose sum does not depend on its order.
template <class T>
__device__ __forceinline__ void sample_row_exact(const SampleParams& P, int64_t row, const RowSettings& S, uint32_t m_key,
                                              int shift, ExactLds& lds) {
  double* const shared = lds.part;
  uint64_t* const mass = lds.mass;
  uint32_t* const count = lds.count;
  uint32_t* const pick = lds.pick;
  uint64_t* const pick_mass = lds.pick_mass;
  const int tid = threadIdx.x;
  const T* x = static_cast<const T*>(P.logits) + row * P.ld;
  auto key_at = [&](int i) { return logit_key(static_cast<float>(dload(P.dbg, 0, kDbgSampleLogits, x + i))); };
  const int V = P.V;
  const float m = key_logit(m_key);
  const double unit = ldexp(1.0, shift);

  // entries with key > edge, or key == edge and position <= edge_pos
  uint32_t edge = 0;
  int edge_pos = V;
  auto inside = [&](uint32_t key, int i) { return key > edge || (key == edge && i <= edge_pos); };
  auto fixed = [&](uint32_t key) { return static_cast<uint64_t>(weight_of(key, m, m_key, S.c) * unit + 0.5); };

  for (int by_mass = 0; by_mass < 2; ++by_mass) {
    if (by_mass ? S.p >= 1.0 : S.k >= static_cast<uint32_t>(V)) continue;
    uint64_t target = S.k;
    if (by_mass) {  // the mass that the prefix has to reach
      if (tid == 0) pick_mass[0] = 0;
      __syncthreads();
      uint64_t w = 0;
      for (int i = tid; i < V; i += kRowThreads) {
        const uint32_t key = key_at(i);
        if (inside(key, i)) w += fixed(key);
      }
      atomicAdd(reinterpret_cast<unsigned long long*>(&pick_mass[0]), static_cast<unsigned long long>(w));
      __syncthreads();
      const double t = S.p * static_cast<double>(pick_mass[0]);
      target = static_cast<uint64_t>(ceil(t));
      if (target == 0) target = 1;
      __syncthreads();
    }
    // the entry at which the prefix reaches the target: its key, digit by digit
    uint32_t prefix = 0;
    uint64_t above = 0;  // reached by the entries of larger keys
    uint32_t ties = 0;
    for (int shift_bits = 24; shift_bits >= 0; shift_bits -= 8) {
      if (tid < kDigits) count[tid] = 0, mass[tid] = 0;
      __syncthreads();
      for (int i = tid; i < V; i += kRowThreads) {
        const uint32_t key = key_at(i);
        if (shift_bits < 24 && (key >> (shift_bits + 8)) != prefix) continue;
        if (!inside(key, i)) continue;
        const uint32_t d = (key >> shift_bits) & 255u;
        atomicAdd(&count[d], 1u);
        if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&mass[d]), static_cast<unsigned long long>(fixed(key)));
      }
      __syncthreads();
      if (tid == 0) {
        uint64_t run = above;
        int at = -1;
        uint64_t at_above = above;
        for (int d = kDigits - 1; d >= 0; --d) {
          const uint64_t w = by_mass ? mass[d] : count[d];
          if (count[d] == 0) continue;
          at = d;
          at_above = run;
          run += w;
          if (run >= target) break;
        }
        pick[0] = static_cast<uint32_t>(at);
        pick[1] = count[at];
        pick_mass[0] = at_above;
      }
      __syncthreads();
      prefix = (prefix << 8) | pick[0];
      ties = pick[1];
      above = pick_mass[0];
      __syncthreads();
    }
    // of the entries equal to that key, the first few positions
    const uint64_t each = by_mass ? max(fixed(prefix), uint64_t(1)) : uint64_t(1);
    const uint64_t need = (target - min(above, target) + each - 1) / each;
    const uint32_t old_edge = edge;
    const int old_pos = edge_pos;
    edge = prefix;
    edge_pos = old_edge == edge ? old_pos : V;
    if (need < ties) {
      const int limit = edge_pos;
      edge_pos = find_position([&](int i) { return i <= limit && key_at(i) == prefix ? 1.0 : 0.0; }, V,
                               static_cast<double>(need) - 0.5, shared);
    }
  }

  auto kept = [&](int i) -> double {
    const uint32_t key = key_at(i);
    if (!inside(key, i)) return 0.0;
    const double w = weight_of(key, m, m_key, S.c);
    return w >= S.q ? w : 0.0;
  };
  double mine = 0.0;
  for (int i = tid; i < V; i += kRowThreads) mine += kept(i);
  const double total = block_sum_f64(mine, shared);
  const int at = find_position(kept, V, S.u * total, shared);
  if (tid == 0) put_draw(P, row, at, kept(at) / total);
}

// ---------------------------------------------------------------------------
// Rows of up to 2^18 entries
// ---------------------------------------------------------------------------

template <class T>
__device__ __forceinline__ float logit_of_bits(uint32_t bits) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
  else return static_cast<float>(__builtin_bit_cast(T, static_cast<uint16_t>(bits)));
}

template <class T>
struct RowView {
  static constexpr int kPer = 16 / sizeof(T);  // elements per piece
  const T* x;
  int lead, V;

  __device__ __forceinline__ RowView(const SampleParams& P, int64_t row)
      : x(static_cast<const T*>(P.logits) + row * P.ld), V(P.V) {
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  }

  // Keys of piece i; 0 (below every logit's key) for elements outside the row.
  __device__ __forceinline__ void piece(const DebugCheck& dbg, int i, uint32_t (&key)[kPer]) const {
    const int first = i * kPer - lead;
    if (first >= 0 && first + kPer <= V) {
      const u32x4 v = dload(dbg, 0, kDbgSampleLogits, reinterpret_cast<const u32x4*>(x + first));
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t w = v[j * sizeof(T) / 4];
        key[j] = logit_key(logit_of_bits<T>(sizeof(T) == 4 ? w : (j & 1) ? w >> 16 : w & 0xffffu));
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int at = first + j;
        key[j] = at >= 0 && at < V ? logit_key(static_cast<float>(dload(dbg, 0, kDbgSampleLogits, x + at))) : 0u;
      }
    }
  }

  __device__ __forceinline__ uint32_t element(const DebugCheck& dbg, int e) const {
    const int at = e - lead;
    return at >= 0 && at < V ? logit_key(static_cast<float>(dload(dbg, 0, kDbgSampleLogits, x + at))) : 0u;
  }
};

// The mass histogram's grid: entry x lies in bin floor(16 x log2(e) / T), a
// monotone function of x; its weight relative to the bin's lower edge is
// 2^(f / 16), f the fraction: exp(y) by Taylor's series to the 6th power, y <=
// ln(2) / 16 (remainder below 6e-14).
__device__ __forceinline__ double bin_weight(double f) {
  const double y = f * (0.69314718055994530942 / 16.0);
  double s = fma(1.0 / 720.0, y, 1.0 / 120.0);
  s = fma(s, y, 1.0 / 24.0);
  s = fma(s, y, 1.0 / 6.0);
  s = fma(s, y, 0.5);
  s = fma(s, y, 1.0);
  return fma(s, y, 1.0);
}

// A histogram word: entries counted from bit 49 up, below it their weights in
// units of 2^-34 (16384 entries of at most 2^(1/16) stay below 2^49). The
// rounding is 2^-35 of a weight, either way: over n entries the sums are off
// by sqrt(n) 2^-35 of a weight, and a draw differs from that of exact sums
// with a probability below 1e-8 at 2^18 entries.
constexpr int kHistShift = 34;
constexpr int kHistCount = 49;
constexpr double kMaxBin = 16777216.0;  // larger |bin| numbers: left to sample_row_exact

__device__ __forceinline__ uint32_t hist_count(uint64_t w) { return static_cast<uint32_t>(w >> kHistCount); }
__device__ __forceinline__ double hist_mass(uint64_t w) {
  return static_cast<double>(w & ((uint64_t(1) << kHistCount) - 1)) * (1.0 / (uint64_t(1) << kHistShift));
}

// One workgroup per chunk of a row. HBM bound where only the maxima are
// wanted; with the masses, the fp64 arithmetic of one exponential per entry
// takes about as long as the reading.
template <class T, int kThreads>
__global__ __launch_bounds__(kThreads) void k_sample_scan(SampleParams P) {
  constexpr int kPer = RowView<T>::kPer;
  constexpr int kPieces = kScanElems / kPer;
  constexpr int kWaves = kThreads / 64;
  constexpr int kLanes = kGroup / kPer;  // lanes that share a group
  __shared__ uint64_t hist[kScanBins];
  __shared__ uint32_t wave_max[kWaves];
  __shared__ double wave_mass[kWaves];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int chunk = blockIdx.x % P.chunks;
  const int64_t row = P.row0 + blockIdx.x / P.chunks;
  const RowView<T> view(P, row);
  const int64_t slot = row * P.chunks + chunk;
  uint32_t key[kPieces][kPer];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) view.piece(P.dbg, chunk * (kThreads * kPieces) + p * kThreads + tid, key[p]);
  const RowSettings S = row_settings(P, row);
  const RowMode mode = row_mode(S, P.V);
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    uint32_t m = key[p][0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) m = max(m, key[p][j]);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, 64)));
    const int g = (chunk * (kThreads * kScanElems) + (p * kThreads + tid) * kPer) / kGroup;
    if (lane % kLanes == 0 && g < P.groups)
      dstore(P.dbg, 5, kDbgSampleWork, P.group_max + row * P.groups + g, m);
    top = max(top, m);
  }
  if (mode == kMaximaOnly) return;
#pragma unroll
  for (int o = 32; o >= kLanes; o >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o, 64)));
  if (lane == 0) wave_max[tid >> 6] = top;
  if (mode == kMassHistogram)
    for (int i = tid; i < kScanBins; i += kThreads) hist[i] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = max(top, wave_max[w]);
  const float m = key_logit(top);
  double sum = 0.0;
  if (mode == kChunkMass) {
    if (top > kMaskedKey) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += weight_of(key[p][j], m, top, S.c);
    }
  } else {
    const double c16 = 16.0 * S.c;
    const double base = floor(static_cast<double>(m) * c16);
    if (top > kMaskedKey && fabs(base) < kMaxBin) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (key[p][j] <= kMaskedKey) continue;
          const double t = static_cast<double>(key_logit(key[p][j])) * c16;
          const double b = floor(t);
          const double d = base - b;
          if (d < kScanBins) {
            const uint64_t w = static_cast<uint64_t>(bin_weight(t - b) * (uint64_t(1) << kHistShift) + 0.5);
            atomicAdd(reinterpret_cast<unsigned long long*>(&hist[static_cast<int>(d)]),
                      static_cast<unsigned long long>((uint64_t(1) << kHistCount) + w));
          } else {
            // 2^-32 of the chunk's largest weight or less: fp32's relative precision is enough
            sum += static_cast<double>(exp2f(static_cast<float>((t - base) * (1.0 / 16.0))));
          }
        }
    }
    __syncthreads();
    for (int i = tid; i < kScanBins; i += kThreads)
      dstore(P.dbg, 5, kDbgSampleWork, P.chunk_hist + slot * kScanBins + i, hist[i]);
  }
  sum = wave_sum_f64(sum);
  if (lane == 0) wave_mass[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int w = 0; w < kWaves; ++w) s += wave_mass[w];
    dstore(P.dbg, 5, kDbgSampleWork, P.chunk_max + slot, top);
    dstore(P.dbg, 5, kDbgSampleWork, P.chunk_mass + slot, s);
  }
}

constexpr int kMaxGroups = (1 << 18) / kGroup + 1;
constexpr int kMaxChunks = (1 << 18) / (256 * kScanElems) + 1;

struct PickLds {
  uint32_t group_max[kMaxGroups];
  union {
    struct {
      uint32_t key[kCandidates];
      int32_t pos[kCandidates];
    } cand;
    uint64_t entry[kCandidates];  // (key, ~position) of the border bin's entries
  };
  union {
    uint32_t sorted[kCandidates];
    uint32_t bins[kRowThreads];
    uint32_t list[kCandidates];  // groups that reach the bound
  };
  double chunk[kMaxChunks + 1];
  double wave_f64[kRowWaves];
  uint32_t wave_u32[kRowWaves];
  uint32_t word[4];
  double value[2];
};

// Exclusive sum of v over the block in thread order; total gets the sum.
__device__ __forceinline__ double block_scan_f64(double v, double* wave, double& total) {
  const int lane = threadIdx.x & 63;
  double incl = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(incl, o, 64);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 63) wave[threadIdx.x >> 6] = incl;
  __syncthreads();
  double base = 0.0, sum = 0.0;
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) {
    if (w == static_cast<int>(threadIdx.x >> 6)) base = sum;
    sum += wave[w];
  }
  total = sum;
  return base + (incl - v);
}

__device__ __forceinline__ uint32_t block_scan_u32(uint32_t v, uint32_t* wave, uint32_t& total) {
  const int lane = threadIdx.x & 63;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = static_cast<uint32_t>(__shfl_up(static_cast<int>(incl), o, 64));
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 63) wave[threadIdx.x >> 6] = incl;
  __syncthreads();
  uint32_t base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) {
    if (w == static_cast<int>(threadIdx.x >> 6)) base = sum;
    sum += wave[w];
  }
  total = sum;
  return base + (incl - v);
}

// Sorts n keys (LDS, room for the next power of two >= 64) in descending order;
// the keys past n are 0.
template <class K>
__device__ void sort_descending(K* a, int n) {
  int size = 64;
  while (size < n) size <<= 1;
  const int tid = threadIdx.x;
  for (int i = n + tid; i < size; i += kRowThreads) a[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int p = tid; p < size / 2; p += kRowThreads) {
        const int i = 2 * p - (p & (j - 1));
        const K x = a[i], y = a[i + j];
        if ((x < y) == ((i & k) == 0)) a[i] = y, a[i + j] = x;
      }
      __syncthreads();
    }
  }
}

// Upper bound on the distance from the largest key for the bins of
// bound_of_kth: exact below 32, then 32 bins per power of two.
__device__ __forceinline__ uint32_t distance_bin(uint32_t d) {
  if (d < 32) return d;
  const int e = 31 - __clz(static_cast<int>(d));
  return static_cast<uint32_t>((e - 4) * 32) + ((d >> (e - 5)) & 31u);
}
__device__ __forceinline__ uint32_t distance_bin_end(uint32_t b) {
  if (b < 32) return b;
  const int e = static_cast<int>(b >> 5) + 4;
  return static_cast<uint32_t>((static_cast<uint64_t>(32 + (b & 31u)) + 1) << (e - 5)) - 1u;
}

// A key that at least k of the row's entries reach: at least k group maxima
// do. kMaskedKey + 1 where fewer than k groups hold an unmasked entry.
__device__ uint32_t bound_of_kth(PickLds& L, int groups, uint32_t m_key, uint32_t k) {
  const int tid = threadIdx.x;
  L.bins[tid] = 0;
  if (tid == 0) L.word[0] = kMaskedKey + 1;
  __syncthreads();
  for (int g = tid; g < groups; g += kRowThreads)
    if (L.group_max[g] > kMaskedKey) atomicAdd(&L.bins[distance_bin(m_key - L.group_max[g])], 1u);
  __syncthreads();
  const uint32_t mine = L.bins[tid];
  uint32_t total;
  const uint32_t before = block_scan_u32(mine, L.wave_u32, total);
  if (before < k && before + mine >= k) {
    const uint32_t d = distance_bin_end(static_cast<uint32_t>(tid));
    L.word[0] = max(kMaskedKey + 1, d < m_key ? m_key - d : 0u);
  }
  __syncthreads();
  const uint32_t bound = L.word[0];
  __syncthreads();
  return bound;
}

// The draw within one chunk: the first position at which base plus the kept
// weights up to it exceeds target; weight(key, position) is 0 for what is not
// kept. Returns the position and its weight to every thread.
template <class T, class Weight>
__device__ int draw_in_chunk(const SampleParams& P, const RowView<T>& view, PickLds& L, int chunk, double base,
                             double target, Weight weight, double& w_at) {
  constexpr int kPer = RowView<T>::kPer;
  const int tid = threadIdx.x;
  const int pieces = P.chunk_elems / kPer;
  if (tid == 0) L.word[0] = 0xffffffffu, L.word[1] = 0;
  for (int p0 = 0; p0 < pieces; p0 += kRowThreads) {
    uint32_t key[kPer];
    double w[kPer], sum = 0.0, total;
    const int piece = chunk * pieces + p0 + tid;
    const bool live = p0 + tid < pieces;
    if (live) view.piece(P.dbg, piece, key);
    int last = -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      w[j] = live ? weight(key[j], piece * kPer - view.lead + j) : 0.0;
      sum += w[j];
      if (w[j] > 0.0) last = j;
    }
    const double before = base + block_scan_f64(sum, L.wave_f64, total);
    if (sum > 0.0) {
      double run = before;
      int at = -1;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        run += w[j];
        if (at < 0 && w[j] > 0.0 && run > target) at = j;
      }
      const uint32_t pos = static_cast<uint32_t>(piece * kPer - view.lead);
      if (at >= 0) atomicMin(&L.word[0], pos + at);
      atomicMax(&L.word[1], pos + last);  // if rounding leaves no such position: the last one kept
    }
    base += total;
    __syncthreads();
    if (L.word[0] != 0xffffffffu) break;
  }
  const int at = static_cast<int>(L.word[0] != 0xffffffffu ? L.word[0] : L.word[1]);
  w_at = weight(logit_key(static_cast<float>(dload(P.dbg, 0, kDbgSampleLogits, view.x + at))), at);
  __syncthreads();
  return at;
}

// The chunk in which the running sum of L.chunk[0 .. n) exceeds target (the
// last one that is not empty if rounding leaves none); base: the sum before it.
__device__ int find_chunk(const PickLds& L, int n, double target, double& base) {
  int at = 0;
  double run = 0.0;
  bool found = false;
  base = 0.0;
  for (int i = 0; i < n; ++i) {
    const double w = L.chunk[i];
    if (!found && w > 0.0) {
      at = i;
      base = run;
      found = run + w > target;
    }
    run += w;
  }
  return at;
}

// Settles a row from what the scan left; false where the border is too wide
// for this route (the same for every thread).
template <class T>
__device__ __forceinline__ bool pick_row(const SampleParams& P, int64_t row, const RowSettings& S,
                                         const RowView<T>& view, uint32_t m_key, PickLds& L) {
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int V = P.V;
  const RowMode mode = row_mode(S, V);
  const float m = key_logit(m_key);
  const int64_t slot = row * P.chunks;
  // the whole row's mass relative to m
  double total = 0.0;
  if (mode == kChunkMass) {
    if (tid < P.chunks) {
      const uint32_t ck = dload(P.dbg, 5, kDbgSampleWork, P.chunk_max + slot + tid);
      const double cm = dload(P.dbg, 5, kDbgSampleWork, P.chunk_mass + slot + tid);
      L.chunk[tid] = ck > kMaskedKey ? cm * weight_of(ck, m, m_key, S.c) : 0.0;
    }
    __syncthreads();
    for (int i = 0; i < P.chunks; ++i) total += L.chunk[i];
    if (S.p >= 1.0 && S.q <= 0.0) {  // no filter: a chunk, then a position in it
      double base, w;
      const double target = S.u * total;
      const int chunk = find_chunk(L, P.chunks, target, base);
      const int at = draw_in_chunk(P, view, L, chunk, base, target,
                                   [&](uint32_t key, int) { return weight_of(key, m, m_key, S.c); }, w);
      if (tid == 0) put_draw(P, row, at, w / total);
      return true;
    }
  }

  // a key that every kept entry reaches
  uint32_t bound = kMaskedKey + 1;
  if (S.k < static_cast<uint32_t>(V)) bound = S.k == 1 ? m_key : bound_of_kth(L, P.groups, m_key, S.k);
  if (S.q > 0.0 && isfinite(m) && (S.p >= 1.0 || S.k >= static_cast<uint32_t>(V))) {
    // w >= q: x >= m + log2(q) / c, taken lower by more than its rounding
    // (top-p after top-k needs the mass of all the k entries: no bound from q then)
    const double lo = static_cast<double>(m) + log2(S.q) / S.c;
    const float low = static_cast<float>(lo - 1e-6 * fabs(lo) - 1e-30);
    bound = max(bound, logit_key(low));
  }
  if (mode == kMassHistogram) {
    const double c16 = 16.0 * S.c;
    const double t_max = static_cast<double>(m) * c16;
    const double base = floor(t_max);
    if (!(fabs(base) < kMaxBin)) return false;
    // bin d (from the top) of the row, and the mass below the last bin
    uint32_t cnt = 0;
    double mass = 0.0, rest = 0.0;
    for (int ch = 0; ch < P.chunks; ++ch) {
      const uint32_t ck = dload(P.dbg, 5, kDbgSampleWork, P.chunk_max + slot + ch);
      if (ck <= kMaskedKey) continue;
      const double cb = floor(static_cast<double>(key_logit(ck)) * c16);
      const double off = base - cb;  // >= 0: the chunk's bins start this much lower
      if (tid < kScanBins) {
        const uint64_t w = dload(P.dbg, 5, kDbgSampleWork, P.chunk_hist + (slot + ch) * kScanBins + tid);
        // added up below through LDS: chunk bin tid is row bin tid + off
        const double d = off + tid;
        if (w) {
          if (d < kScanBins) {
            if (off == 0.0) cnt += hist_count(w), mass += hist_mass(w);
          } else {
            rest += hist_mass(w) * exp2_neg(-d * (1.0 / 16.0));
          }
        }
        const int src = tid - static_cast<int>(off < kScanBins ? off : kScanBins);
        if (off > 0.0 && off < kScanBins && src >= 0) {
          const uint64_t v = dload(P.dbg, 5, kDbgSampleWork, P.chunk_hist + (slot + ch) * kScanBins + src);
          cnt += hist_count(v), mass += hist_mass(v);
        }
      }
      if (tid == kScanBins)
        rest += dload(P.dbg, 5, kDbgSampleWork, P.chunk_mass + slot + ch) * exp2_neg(-off * (1.0 / 16.0));
    }
    const double scaled = mass * exp2_neg(-tid * (1.0 / 16.0));  // relative to 2^(base / 16)
    double in_bins, rest_all;
    const double above = block_scan_f64(scaled, L.wave_f64, in_bins);
    block_scan_f64(rest, L.wave_f64, rest_all);
    uint32_t counted;
    const uint32_t cnt_above = block_scan_u32(cnt, L.wave_u32, counted);
    const double whole = in_bins + rest_all;
    const double target = S.p * whole;
    if (tid == 0) L.word[1] = 0xffffffffu;
    __syncthreads();
    if (cnt > 0 && above < target && above + scaled >= target) {
      atomicMin(&L.word[1], static_cast<uint32_t>(tid));
    }
    __syncthreads();
    const uint32_t border = L.word[1];
    if (border == 0xffffffffu) return false;  // below the bins
    if (static_cast<uint32_t>(tid) == border) L.word[2] = cnt, L.word[3] = cnt_above, L.value[0] = above;
    __syncthreads();
    const uint32_t in_border = L.word[2];
    const uint32_t n_above = L.word[3];
    const double mass_above = L.value[0];
    __syncthreads();
    const double edge_bin = base - static_cast<double>(border);
    if (n_above + in_border <= kCandidates) {
      total = whole * exp2_neg((base - t_max) * (1.0 / 16.0));
      const double lo = edge_bin / c16;
      const float low = static_cast<float>(lo - 1e-6 * fabs(lo) - 1e-30);
      bound = max(bound, logit_key(low));
    } else {
      // Too many entries are kept to hold them: only the border bin's are
      // gathered and ordered; the bins above it are kept whole.
      if (in_border > kCandidates) return false;
      if (tid == 0) L.word[0] = 0;
      __syncthreads();
      constexpr int kPer = RowView<T>::kPer;
      const int pieces = (view.lead + V + kPer - 1) / kPer;
      for (int i = tid; i < pieces; i += kRowThreads) {
        uint32_t key[kPer];
        view.piece(P.dbg, i, key);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (key[j] <= kMaskedKey) continue;
          if (floor(static_cast<double>(key_logit(key[j])) * c16) == edge_bin) {
            const uint32_t n = atomicAdd(&L.word[0], 1u);
            if (n < kCandidates)
              L.entry[n] = (static_cast<uint64_t>(key[j]) << 32) |
                           (0xffffffffu - static_cast<uint32_t>(i * kPer - view.lead + j));
          }
        }
      }
      __syncthreads();
      const int n = static_cast<int>(in_border);
      sort_descending(L.entry, n);
      auto weight = [&](uint32_t key) {  // relative to 2^(base / 16)
        const double t = static_cast<double>(key_logit(key)) * c16 - base;
        return t > 0.0 ? 1.0 / exp2_neg(-t * (1.0 / 16.0)) : exp2_neg(t * (1.0 / 16.0));
      };
      // the last kept entry of the bin: the last before which less than the target lies
      if (tid == 0) L.word[0] = 0;
      double run = mass_above;
      for (int i0 = 0; i0 < n; i0 += kRowThreads) {
        const int i = i0 + tid;
        const double w = i < n ? weight(static_cast<uint32_t>(L.entry[i] >> 32)) : 0.0;
        double sum;
        const double before = run + block_scan_f64(w, L.wave_f64, sum);
        if (i < n && before < target) atomicMax(&L.word[0], static_cast<uint32_t>(i));
        run += sum;
      }
      __syncthreads();
      const int last = static_cast<int>(L.word[0]);
      const uint64_t edge = L.entry[last];
      const uint32_t edge_key = static_cast<uint32_t>(edge >> 32);
      const int edge_pos = static_cast<int>(0xffffffffu - static_cast<uint32_t>(edge));
      // each chunk's kept mass: its bins above the border, and its kept entries of the border bin
      for (int ch = wave; ch < P.chunks; ch += kRowWaves) {
        const uint32_t ck = dload(P.dbg, 5, kDbgSampleWork, P.chunk_max + slot + ch);
        double s = 0.0;
        if (ck > kMaskedKey) {
          const double off = base - floor(static_cast<double>(key_logit(ck)) * c16);
          for (int d = lane; d < kScanBins && off + d < border; d += 64) {
            const uint64_t w = dload(P.dbg, 5, kDbgSampleWork, P.chunk_hist + (slot + ch) * kScanBins + d);
            if (w) s += hist_mass(w) * exp2_neg(-(off + d) * (1.0 / 16.0));
          }
          for (int i = lane; i <= last; i += 64) {
            const uint64_t en = L.entry[i];
            const int e = static_cast<int>(0xffffffffu - static_cast<uint32_t>(en)) + view.lead;
            if (e / P.chunk_elems == ch) s += weight(static_cast<uint32_t>(en >> 32));
          }
        }
        s = wave_sum_f64(s);
        if (lane == 0) L.chunk[ch] = s;
      }
      __syncthreads();
      double kept = 0.0, before, w;
      for (int i = 0; i < P.chunks; ++i) kept += L.chunk[i];
      const double goal = S.u * kept;
      const int chunk = find_chunk(L, P.chunks, goal, before);
      const int at = draw_in_chunk(P, view, L, chunk, before, goal,
                                   [&](uint32_t key, int pos) {
                                     const bool in = key > edge_key || (key == edge_key && pos <= edge_pos);
                                     return in ? weight(key) : 0.0;
                                   }, w);
      if (tid == 0) put_draw(P, row, at, w / kept);
      return true;
    }
  }

  // The groups that reach the bound, in order, and their entries that do: the
  // candidates, in order of position.
  uint32_t n_list;
  {
    const int per = (P.groups + kRowThreads - 1) / kRowThreads;
    const int g0 = min(tid * per, P.groups), g1 = min(g0 + per, P.groups);
    uint32_t mine = 0;
    for (int g = g0; g < g1; ++g) mine += L.group_max[g] >= bound;
    uint32_t at = block_scan_u32(mine, L.wave_u32, n_list);
    if (n_list > kCandidates) return false;
    for (int g = g0; g < g1; ++g)
      if (L.group_max[g] >= bound) L.list[at++] = static_cast<uint32_t>(g);
  }
  __syncthreads();
  const int per_wave = (static_cast<int>(n_list) + kRowWaves - 1) / kRowWaves;
  const int l0 = min(wave * per_wave, static_cast<int>(n_list));
  const int l1 = min(l0 + per_wave, static_cast<int>(n_list));
  uint32_t found = 0;
#pragma unroll 4
  for (int l = l0; l < l1; ++l) {
    const uint32_t key = view.element(P.dbg, static_cast<int>(L.list[l]) * kGroup + lane);
    found += __popcll(__ballot(key >= bound));
  }
  uint32_t n_cand;
  uint32_t put = block_scan_u32(lane == 0 ? found : 0u, L.wave_u32, n_cand);
  if (n_cand > kCandidates) return false;
  put = __shfl(static_cast<int>(put), 0, 64);
#pragma unroll 4
  for (int l = l0; l < l1; ++l) {
    const int e = static_cast<int>(L.list[l]) * kGroup + lane;
    const uint32_t key = view.element(P.dbg, e);
    const uint64_t hit = __ballot(key >= bound);
    const uint32_t at = put + __popcll(hit & ((uint64_t(1) << lane) - 1));
    if (key >= bound) {
      L.cand.key[at] = key;
      L.cand.pos[at] = e - view.lead;
    }
    put += __popcll(hit);
  }
  __syncthreads();
  const int n = static_cast<int>(n_cand);
  for (int i = tid; i < n; i += kRowThreads) L.sorted[i] = L.cand.key[i];
  sort_descending(L.sorted, n);
  // the kept prefix of the sorted candidates
  const int kk = static_cast<int>(min(S.k, static_cast<uint32_t>(n)));
  auto weight = [&](uint32_t key) { return weight_of(key, m, m_key, S.c); };
  double mass = total;
  if (S.p < 1.0 && S.k < static_cast<uint32_t>(V)) {
    double s = 0.0;
    for (int i = tid; i < kk; i += kRowThreads) s += weight(L.sorted[i]);
    block_scan_f64(s, L.wave_f64, mass);
  }
  const double target = S.p * mass;
  if (tid == 0) L.word[0] = 0;
  double run = 0.0;
  for (int i0 = 0; i0 < kk; i0 += kRowThreads) {
    const int i = i0 + tid;
    const double w = i < kk ? weight(L.sorted[i]) : 0.0;
    double sum;
    const double before = run + block_scan_f64(w, L.wave_f64, sum);
    if (i < kk && (S.p >= 1.0 || before < target) && w >= S.q) atomicMax(&L.word[0], static_cast<uint32_t>(i));
    run += sum;
  }
  __syncthreads();
  const int last = static_cast<int>(L.word[0]);
  const uint32_t edge = L.sorted[last];
  if (tid == 0) L.word[1] = 0;
  __syncthreads();
  for (int i = tid; i <= last; i += kRowThreads)
    if (L.sorted[i] == edge) atomicAdd(&L.word[1], 1u);
  __syncthreads();
  const uint32_t quota = L.word[1];  // of the entries equal to the border's, the first this many positions
  // the draw: thread t holds candidates t * per .. in order of position
  const int per = (n + kRowThreads - 1) / kRowThreads;
  const int c0 = min(tid * per, n), c1 = min(c0 + per, n);
  uint32_t ties = 0, all_ties;
  for (int i = c0; i < c1; ++i) ties += L.cand.key[i] == edge;
  const uint32_t ties_before = block_scan_u32(ties, L.wave_u32, all_ties);
  auto kept = [&](int i, uint32_t& t) {
    const uint32_t key = L.cand.key[i];
    if (key < edge) return 0.0;
    if (key == edge && t++ >= quota) return 0.0;
    return weight(key);
  };
  double sum = 0.0, whole;
  uint32_t t = ties_before;
  for (int i = c0; i < c1; ++i) sum += kept(i, t);
  const double before = block_scan_f64(sum, L.wave_f64, whole);
  const double goal = S.u * whole;
  if (tid == 0) L.word[2] = 0xffffffffu, L.word[3] = 0;
  __syncthreads();
  double acc = before;
  t = ties_before;
  for (int i = c0; i < c1; ++i) {
    const double w = kept(i, t);
    acc += w;
    if (w > 0.0) {
      if (acc > goal) atomicMin(&L.word[2], static_cast<uint32_t>(i));
      atomicMax(&L.word[3], static_cast<uint32_t>(i));
    }
  }
  __syncthreads();
  if (tid == 0) {
    const uint32_t i = L.word[2] != 0xffffffffu ? L.word[2] : L.word[3];
    put_draw(P, row, L.cand.pos[i], weight(L.cand.key[i]) / whole);
  }
  return true;
}

// One workgroup per row, after k_sample_scan. Latency bound: a chain of short
// steps over LDS, with one dependent read of the groups that reach the bound.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_sample_pick(SampleParams P, int shift) {
  __shared__ union {
    PickLds pick;
    ExactLds exact;
  } lds;
  PickLds& L = lds.pick;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int64_t row = P.row0 + blockIdx.x;
  uint32_t m_key = 0;
  for (int g = tid; g < P.groups; g += kRowThreads) {
    const uint32_t v = dload(P.dbg, 5, kDbgSampleWork, P.group_max + row * P.groups + g);
    L.group_max[g] = v;
    m_key = max(m_key, v);
  }
  const RowSettings S = row_settings(P, row);
  const RowView<T> view(P, row);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m_key = max(m_key, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m_key), o, 64)));
  if (lane == 0) L.wave_u32[wave] = m_key;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) m_key = max(m_key, L.wave_u32[w]);
  __syncthreads();
  if (!S.valid || m_key <= kMaskedKey) {
    if (tid == 0) put_none(P, row);
    return;
  }
  if (pick_row<T>(P, row, S, view, m_key, L)) return;
  __syncthreads();
  sample_row_exact<T>(P, row, S, m_key, shift, lds.exact);
}

// Rows longer than the scan takes: the largest key, then sample_row_exact.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_sample_long(SampleParams P, int shift) {
  __shared__ ExactLds lds;
  const int tid = threadIdx.x;
  const int64_t row = P.row0 + blockIdx.x;
  const RowSettings S = row_settings(P, row);
  const RowView<T> view(P, row);
  uint32_t m_key = 0;
  for (int i = tid; i < P.V; i += kRowThreads) m_key = max(m_key, view.element(P.dbg, view.lead + i));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m_key = max(m_key, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m_key), o, 64)));
  if ((tid & 63) == 0) lds.count[tid >> 6] = m_key;
  __syncthreads();
  for (int w = 0; w < kRowWaves; ++w) m_key = max(m_key, lds.count[w]);
  __syncthreads();
  if (!S.valid || m_key <= kMaskedKey) {
    if (tid == 0) put_none(P, row);
    return;
  }
  sample_row_exact<T>(P, row, S, m_key, shift, lds);
}

template <class T>
static void launch_sample_of(const SamplePlan& p, SampleParams P, int shift, hipStream_t st) {
  // grid x block stays below 2^32 threads
  const int64_t per_row = p.route == kSampleScan ? p.chunks : 1;
  const int64_t rows_max = std::max<int64_t>(1, (int64_t(1) << 21) / per_row);
  const double bytes = static_cast<double>(p.N) * p.V * sizeof(T);
  for (int64_t r = 0; r < p.N; r += rows_max) {
    const int64_t rows = std::min(p.N - r, rows_max);
    P.row0 = r;
    if (p.route == kSampleLong) {
      TraceScope ts(st, "sample_long", 0.0, bytes);
      hipLaunchKernelGGL(k_sample_long<T>, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, st, P, shift);
      continue;
    }
    {
      TraceScope ts(st, "sample_scan", 0.0, bytes);
      const dim3 grid(static_cast<unsigned>(rows * p.chunks));
      if (p.chunk_elems == 256 * kScanElems)
        hipLaunchKernelGGL((k_sample_scan<T, 256>), grid, dim3(256), 0, st, P);
      else
        hipLaunchKernelGGL((k_sample_scan<T, 1024>), grid, dim3(1024), 0, st, P);
    }
    TraceScope ts(st, "sample_pick", 0.0, 4.0 * p.N * p.groups);
    hipLaunchKernelGGL(k_sample_pick<T>, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, st, P, shift);
  }
}

hipError_t launch_sample(const SamplePlan& p, const SampleArgs& a, hipStream_t st) {
  SampleParams P;
  P.logits = a.logits, P.ld = p.ld;
  P.ids = a.ids, P.ld_ids = p.ld_ids;
  P.u = a.u, P.set = a.params;
  P.token = a.token, P.logprob = a.logprob;
  P.V = static_cast<int32_t>(p.V);
  P.groups = static_cast<int32_t>(p.groups);
  P.chunks = static_cast<int32_t>(p.chunks);
  P.chunk_elems = static_cast<int32_t>(p.chunk_elems);
  P.group_max = reinterpret_cast<uint32_t*>(a.ws + p.off_group_max);
  P.chunk_max = reinterpret_cast<uint32_t*>(a.ws + p.off_chunk_max);
  P.chunk_mass = reinterpret_cast<double*>(a.ws + p.off_chunk_mass);
  P.chunk_hist = reinterpret_cast<uint64_t*>(a.ws + p.off_chunk_hist);
  const uint64_t n = static_cast<uint64_t>(p.N);
  P.dbg = make_debug_check(reinterpret_cast<uint32_t*>(a.ws + kDebugWordOffset),
                           {{a.logits, ((n - 1) * p.ld + p.V) * type_bytes(p.type)},
                            {a.ids, a.ids ? ((n - 1) * p.ld_ids + p.V) * 4 : 0},
                            {a.u, n * 4},
                            {a.token, n * 4},
                            {a.logprob, a.logprob ? n * 4 : 0},
                            {a.ws + 256, p.bytes - 256}});
  // V weights of at most 2^shift each stay below 2^63
  int shift = 46;
  while ((p.V >> (62 - shift)) > 0) --shift;
  if (p.type == FKL_F32) launch_sample_of<float>(p, P, shift, st);
  else if (p.type == FKL_BF16) launch_sample_of<__bf16>(p, P, shift, st);
  else launch_sample_of<_Float16>(p, P, shift, st);
  return hipGetLastError();
}

}  // namespace fkl
