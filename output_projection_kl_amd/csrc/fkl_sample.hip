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
// The routes, by the row length:
//   up to 1024 entries: k_sample_short, one wave per row, the row in registers.
//   up to 8192, for up to one row per CU: k_sample_row, the next route's two
//     kernels in one.
//   up to 2^20: k_sample_scan reads the logits once, spread over all CUs, and
//     leaves per row the largest logit of every 16, 64 or 256 entries and, where the
//     filters need it, the mass or a mass histogram of every chunk;
//     k_sample_pick, one workgroup per row, bounds the border from those,
//     reads again only the groups that reach the bound (or one chunk), and
//     settles the border and the draw exactly among them.
//   longer rows, and rows whose border the bound leaves too wide (thousands of
//     equal logits, thousands of entries kept by top-k): sample_row_exact, one
//     workgroup per row, radix selection over the row itself.
#include <algorithm>
#include <type_traits>

#include "fkl_decode.h"
#include "fkl_device.h"

namespace fkl {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

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

// Cross-lane moves within a wave by DPP: lane i receives the value of the lane
// that CTRL names, 0 where there is none or its row is not in ROWS.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{dpp<CTRL, ROWS>(w[0]), dpp<CTRL, ROWS>(w[1])});
}

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint64_t dpp(uint64_t v) {
  return __builtin_bit_cast(uint64_t, dpp<CTRL, ROWS>(__builtin_bit_cast(double, v)));
}

__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ double from_lane(double v, int lane) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{from_lane(w[0], lane), from_lane(w[1], lane)});
}

__device__ __forceinline__ uint64_t from_lane(uint64_t v, int lane) {
  return __builtin_bit_cast(uint64_t, from_lane(__builtin_bit_cast(double, v), lane));
}

// Inclusive running sums over the wave: within each row of 16 lanes by shifts
// of 1, 2, 4 and 8, then the row ends carried over (lane 15 of a row into the
// next, lane 31 into the upper half).
template <class V>
__device__ __forceinline__ V wave_scan(V v) {
  v += dpp<0x111>(v);
  v += dpp<0x112>(v);
  v += dpp<0x114>(v);
  v += dpp<0x118>(v);
  v += dpp<0x142, 0xa>(v);
  v += dpp<0x143, 0xc>(v);
  return v;
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp<0x111>(v));
  v = max(v, dpp<0x112>(v));
  v = max(v, dpp<0x114>(v));
  v = max(v, dpp<0x118>(v));
  v = max(v, dpp<0x142, 0xa>(v));
  v = max(v, dpp<0x143, 0xc>(v));
  return from_lane(v, 63);
}

__device__ __forceinline__ double wave_sum_f64(double v) { return from_lane(wave_scan(v), 63); }

// The value of lane (this lane ^ X).
template <int X>
__device__ __forceinline__ uint32_t xor_lane(uint32_t v) {
  static_assert(X == 1 || X == 2 || X == 4 || X == 8 || X == 16 || X == 32, "one bit");
  if constexpr (X == 1) return dpp<0xb1>(v);                 // pairs swapped
  else if constexpr (X == 2) return dpp<0x4e>(v);            // pairs of pairs swapped
  else if constexpr (X == 4) return dpp<0x1b>(dpp<0x141>(v));  // mirrored in eights, then in fours
  else if constexpr (X == 8) return dpp<0x128>(v);           // rotated by 8 of 16
  else if constexpr (X == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? r[0] : r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & 32) ? r[0] : r[1];
  }
}

template <int X>
__device__ __forceinline__ float xor_lane_f32(float v) {
  return __uint_as_float(xor_lane<X>(__float_as_uint(v)));
}

// 2^t in fp64: t = n + f with |f| <= 1/2, the Taylor series of exp(f ln 2) to
// the 12th power (remainder below 0.3466^13 / 13! = 1.7e-16). 0 below 2^-1022.
__device__ __forceinline__ double exp2_f64(double t) {
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

// 2^(t / 8): t = b + f with b the nearest integer (found by adding and
// subtracting 1.5 * 2^52, whose sum holds b in its low word; |t| < 2^31) and
// |f| <= 1/2; 2^(f / 8) by Taylor's series to the 6th power (remainder below
// 0.0434^7 / 7! = 6e-14). The scan takes one of these of every entry: the
// series' coefficients are kept in scalar registers, which the compiler would
// otherwise copy to vector registers for each entry (a third more instructions).
struct Eighths {
  int b;
  double f;
  __device__ __forceinline__ explicit Eighths(double t) {
    const double r = t + 6755399441055744.0;
    b = static_cast<int>(__double2loint(r));
    f = t - (r - 6755399441055744.0);
  }
};

struct EighthSeries {
  double c[6];
  __device__ __forceinline__ EighthSeries() {
    constexpr double g = 0.69314718055994530942 / 8.0;
    c[0] = g, c[1] = g * g / 2.0, c[2] = g * g * g / 6.0, c[3] = g * g * g * g / 24.0;
    c[4] = g * g * g * g * g / 120.0, c[5] = g * g * g * g * g * g / 720.0;
#pragma unroll
    for (int i = 0; i < 6; ++i) asm("" : "+s"(c[i]));
  }
  __device__ __forceinline__ double operator()(double f) const {
    double s = fma(c[5], f, c[4]);
#pragma unroll
    for (int i = 3; i >= 0; --i) s = fma(s, f, c[i]);
    return fma(s, f, 1.0);
  }
};

// log(w / total) for 0 < w <= total, in fp64: the exponents' difference, and
// the mantissas' ratio (brought within sqrt(2) of 1) by 2 atanh((a - b) / (a +
// b)), whose series to the 17th power leaves less than 0.1716^19 / 19 = 2e-16.
__device__ __forceinline__ double log_ratio(double w, double total) {
  double a = __builtin_amdgcn_frexp_mant(w);
  const double b = __builtin_amdgcn_frexp_mant(total);
  int e = __builtin_amdgcn_frexp_exp(w) - __builtin_amdgcn_frexp_exp(total);
  if (a > 1.4142135623730951 * b) a *= 0.5, ++e;
  else if (1.4142135623730951 * a < b) a *= 2.0, --e;
  const double s = (a - b) / (a + b);
  const double z = s * s;
  double t = 1.0 / 17.0;
#pragma unroll
  for (int i = 15; i > 0; i -= 2) t = fma(t, z, 1.0 / i);
  return fma(static_cast<double>(e), 0.69314718055994530942, 2.0 * s * t);
}

// Geometry of the scan. A row is read in 16-byte pieces at 16-byte aligned
// addresses: element e of the row's pieces is position e - lead, lead the
// elements between the aligned address and the row's start.
constexpr int kScanElems = 16;             // elements per thread of a scan workgroup
constexpr int kScanBins = 512;             // mass histogram: bins of 1/8 bit below the chunk's maximum
constexpr int kCandidates = 4096;          // entries that k_sample_pick settles in LDS,
constexpr int kWaveCandidates = 128;       // and how many of them by one wave
constexpr int kFlatRow = 1024;             // kept entries above which only the border's are gathered,
constexpr int kFlatEntries = 6144;         // at most this many of them
constexpr int kShortRow = 1024;

struct SampleParams {
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  int64_t ld_ids;
  const float* u;
  fkl_sample_params set;
  double c;  // log2(e) / T of the shared temperature
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
  int32_t groups, group_shift, chunks, chunk_elems;
  DebugCheck dbg;  // debug build: span 0 = logits, 1 = ids, 2 = u, 3 = token, 4 = logprob
};

// One row's settings in the form that the kernels use.
struct RowSettings {
  bool valid;
  double c;     // log2(e) / T
  uint32_t k;   // entries kept at most; 2^31 - 1 when off
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
  s.k = first ? 1u : (k <= 0 || k >= P.V) ? 0x7fffffffu : static_cast<uint32_t>(k);
  s.c = !(T > 0.0f) ? 1.0 : P.set.temperature_rows ? 1.4426950408889634074 / static_cast<double>(T) : P.c;
  s.p = first || !(p < 1.0f) ? 1.0 : static_cast<double>(p);
  s.q = first || !(q > 0.0f) ? 0.0 : static_cast<double>(q);
  s.u = u > 0.0f ? static_cast<double>(fminf(u, 1.0f)) : 0.0;
  return s;
}

// What the scan leaves for a row beside the maxima: nothing where top-k or
// min-p bound the border by themselves or a filtered row's entries can all be
// held (64 x 2000 with top-k 50 and top-p: 10.5 us instead of 16 by
// histograms), each chunk's mass where the whole row's mass counts, each chunk's
// mass histogram where top-p alone decides, or top-k with too many entries for
// the group maxima to bound it well.
enum RowMode { kMaximaOnly, kChunkMass, kMassHistogram };

__device__ __forceinline__ RowMode row_mode(const RowSettings& s, const SampleParams& P) {
  if (P.V <= kCandidates && (s.k < static_cast<uint32_t>(P.V) || s.p < 1.0)) return kMaximaOnly;  // all can be candidates
  if (s.k < static_cast<uint32_t>(P.V)) return s.k > static_cast<uint32_t>(P.groups) / 4 ? kMassHistogram : kMaximaOnly;
  if (s.p < 1.0) return s.q > 0.0 ? kChunkMass : kMassHistogram;
  return s.q > 0.0 ? kMaximaOnly : kChunkMass;
}

// Weight of an entry relative to the row's largest logit m.
__device__ __forceinline__ double weight_of(uint32_t key, float m, uint32_t m_key, double c) {
  if (key == m_key) return 1.0;
  if (key <= kMaskedKey) return 0.0;
  return exp2_f64((static_cast<double>(key_logit(key)) - static_cast<double>(m)) * c);
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
      const double incl = wave_scan(mine);
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

__device__ __forceinline__ void put_draw(const SampleParams& P, int64_t row, int at, double w, double total) {
  const int32_t id = P.ids ? dload(P.dbg, 1, kDbgSampleLogits, P.ids + row * P.ld_ids + at) : at;
  dstore(P.dbg, 3, kDbgSampleOut, P.token + row, id);
  if (P.logprob) dstore(P.dbg, 4, kDbgSampleOut, P.logprob + row, static_cast<float>(log_ratio(w, total)));
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
// units of 2^-shift, whose sum does not depend on its order. Eight to ten reads
// of the row by one CU, and LDS atomics: 0.75 ms for 128256 equal logits and
// top-p, 0.9 to 1.3 ms for top-k 5000 with top-p, whatever the number of rows up
// to one per CU.
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
      for (int i0 = 0; i0 < V; i0 += kRowThreads) {  // the same for all lanes: they vote
        const int i = i0 + tid;
        const uint32_t key = i < V ? key_at(i) : 0u;
        bool left = i < V && (shift_bits == 24 || (key >> (shift_bits + 8)) == prefix) && inside(key, i);
        const uint32_t d = (key >> shift_bits) & 255u;
        const uint64_t units = left && by_mass ? fixed(key) : 0;
        // the first digits are shared by most of a wave's entries, and atomics
        // of many lanes on one address are carried out one after the other: the
        // first few digits met are added up across the wave
        for (int t = 0; t < 3; ++t) {
          const uint64_t todo = __ballot(left);
          if (todo == 0) break;
          const int lead = __ffsll(static_cast<long long>(todo)) - 1;
          const bool mine = left && d == from_lane(d, lead);
          const uint64_t same = __ballot(mine);
          const uint64_t sum = by_mass ? from_lane(wave_scan(mine ? units : uint64_t(0)), 63) : 0;
          if ((tid & 63) == lead) {
            atomicAdd(&count[d], static_cast<uint32_t>(__popcll(same)));
            if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&mass[d]), static_cast<unsigned long long>(sum));
          }
          left = left && !mine;
        }
        if (left) {
          atomicAdd(&count[d], 1u);
          if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&mass[d]), static_cast<unsigned long long>(units));
        }
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
  if (tid == 0) put_draw(P, row, at, kept(at), total);
}

// ---------------------------------------------------------------------------
// Rows of up to 2^20 entries
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

  // Piece i as it lies in memory; -inf in place of elements outside the row.
  __device__ __forceinline__ u32x4 raw(const DebugCheck& dbg, int i) const {
    const int first = i * kPer - lead;
    if (first >= 0 && first + kPer <= V) return dload(dbg, 0, kDbgSampleLogits, reinterpret_cast<const u32x4*>(x + first));
    u32x4 v;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int at = first + j;
      const T e = at >= 0 && at < V ? dload(dbg, 0, kDbgSampleLogits, x + at) : static_cast<T>(-INFINITY);
      if constexpr (sizeof(T) == 4) v[j] = __builtin_bit_cast(uint32_t, e);
      else if (j & 1) v[j / 2] |= static_cast<uint32_t>(__builtin_bit_cast(uint16_t, e)) << 16;
      else v[j / 2] = __builtin_bit_cast(uint16_t, e);
    }
    return v;
  }

  __device__ __forceinline__ bool is_whole(int i) const { return i * kPer >= lead && (i + 1) * kPer - lead <= V; }

  // Piece i where all of it is inside the row, some other one where it is not
  // (read in any case: no branch to wait in).
  __device__ __forceinline__ u32x4 whole(const DebugCheck& dbg, int i) const {
    const int in = min(max(i, (lead + kPer - 1) / kPer), (lead + V) / kPer - 1);
    return dload(dbg, 0, kDbgSampleLogits, reinterpret_cast<const u32x4*>(x + (in * kPer - lead)));
  }

  // Pieces i0 + tid + b * stride, b < N, for a block of `stride` threads: all
  // inside the row but for the first and last such batches, which alone look at
  // every piece (a load behind a branch of its own waits there).
  // ONCE: with the hint that they are not asked for again.
  template <int N, bool ONCE = false>
  __device__ __forceinline__ void batch(const DebugCheck& dbg, int i0, int stride, u32x4 (&v)[N]) const {
    const int first = i0 + static_cast<int>(threadIdx.x);
    if (i0 * kPer - lead >= 0 && (i0 + N * stride) * kPer - lead <= V) {
#pragma unroll
      for (int b = 0; b < N; ++b) {
        const u32x4* const at = reinterpret_cast<const u32x4*>(x + ((first + b * stride) * kPer - lead));
        if constexpr (!ONCE) v[b] = dload(dbg, 0, kDbgSampleLogits, at);
        else v[b] = dcheck_range(dbg, 0, kDbgSampleLogits, at, 16) ? __builtin_nontemporal_load(at) : u32x4{0, 0, 0, 0};
      }
    } else {
#pragma unroll
      for (int b = 0; b < N; ++b) v[b] = raw(dbg, first + b * stride);
    }
  }

  static __device__ __forceinline__ float logit(const u32x4& v, int j) {
    const uint32_t w = v[j * sizeof(T) / 4];
    return logit_of_bits<T>(sizeof(T) == 4 ? w : (j & 1) ? w >> 16 : w & 0xffffu);
  }

  // The same as logits.
  __device__ __forceinline__ void logits(const DebugCheck& dbg, int i, float (&v)[kPer]) const {
    const u32x4 w = raw(dbg, i);
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = logit(w, j);
  }

  __device__ __forceinline__ uint32_t element(const DebugCheck& dbg, int e) const {
    const int at = e - lead;  // before the row for a negative e
    const int in = min(max(at, 0), V - 1);  // read in any case: no branch to wait in
    const uint32_t key = logit_key(static_cast<float>(dload(dbg, 0, kDbgSampleLogits, x + in)));
    return at == in ? key : 0u;
  }
};

// The mass histogram's grid: entry x lies in bin rint(8 x log2(e) / T), a
// monotone function of x, with the weight 2^(f / 8) relative to the bin's
// centre. A histogram word holds the number of entries from bit 49 up, and
// below it their weights in units of 2^-34 (16384 entries of at most 2^(1/16)
// stay below 2^49). The rounding is 2^-35 of a weight either way: over n
// entries the sums are off by sqrt(n) 2^-35 of a weight, and a draw differs
// from that of exact sums with a probability below 1e-8.
// Integer sums do not depend on their order.
constexpr int kHistShift = 34;
constexpr int kHistCount = 49;
// Rows that the grid does not fit are left to sample_row_exact: bins beyond
// 2^24, or so wide that the last one's lower end is beyond fp32.
__device__ __forceinline__ bool grid_fits(double base, double c8) { return fabs(base) < 16777216.0 && c8 > 1e-30; }

__device__ __forceinline__ uint32_t hist_count(uint64_t w) { return static_cast<uint32_t>(w >> kHistCount); }
__device__ __forceinline__ uint64_t hist_units(uint64_t w) { return w & ((uint64_t(1) << kHistCount) - 1); }
__device__ __forceinline__ double units_mass(uint64_t units) {
  return static_cast<double>(units) * (1.0 / (uint64_t(1) << kHistShift));
}

// One entry's histogram word: its weight is rounded to units by adding 1.5 *
// 2^18, whose last place is 2^-34.
__device__ __forceinline__ uint64_t hist_word(const EighthSeries& power, const Eighths& x) {
  constexpr uint64_t kBits = 0x4118000000000000ull;  // of 1.5 * 2^18
  return static_cast<uint64_t>(__double_as_longlong(power(x.f) + 393216.0)) +
         ((uint64_t(1) << kHistCount) - kBits);
}

// One workgroup per chunk of a row. HBM bound where only the maxima are
// wanted; with the masses, one fp64 exponential per entry (about 20 vector
// instructions, and an LDS atomic for the histogram) takes about as long as the
// reading. 512 x 201088 fp32 with settings of every kind: 61 us, 6.7 TB/s; 64 x
// 128256 bf16: 3 us for the maxima (5 TB/s, the launch's own time included), 11
// us for the histograms.
template <int kThreads>
struct ScanLds {
  uint64_t hist[kScanBins];
  double eighth[8];
  float wave_top[kThreads / 64];
  double wave_mass[kThreads / 64];
};

template <class T, int kThreads, bool ONCE>
__device__ __forceinline__ void scan_chunk(const SampleParams& P, int64_t row, int chunk, ScanLds<kThreads>& L) {
  constexpr int kPer = RowView<T>::kPer;
  constexpr int kPieces = kScanElems / kPer;
  constexpr int kWaves = kThreads / 64;
  uint64_t* const hist = L.hist;
  double* const eighth = L.eighth;
  float* const wave_top = L.wave_top;
  double* const wave_mass = L.wave_mass;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const RowView<T> view(P, row);
  const int64_t slot = row * P.chunks + chunk;
  u32x4 held[kPieces];
  view.template batch<kPieces, ONCE>(P.dbg, chunk * (kThreads * kPieces), kThreads, held);
  float x[kPieces][kPer];
#pragma unroll
  for (int p = 0; p < kPieces; ++p)
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[p][j] = view.logit(held[p], j);
  const RowSettings S = row_settings(P, row);
  const RowMode mode = row_mode(S, P);
  float top = -INFINITY;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    float m = -INFINITY;  // a NaN is no maximum
#pragma unroll
    for (int j = 0; j < kPer; ++j) m = fmaxf(m, x[p][j]);
    // the maximum of 16, then of 64 consecutive elements
    const int e = chunk * (kThreads * kScanElems) + (p * kThreads + tid) * kPer;
    m = fmaxf(m, xor_lane_f32<1>(m));
    if constexpr (kPer == 4) m = fmaxf(m, xor_lane_f32<2>(m));
    if (P.group_shift == 4 && e % 16 == 0 && e / 16 < P.groups)
      dstore(P.dbg, 5, kDbgSampleWork, P.group_max + row * P.groups + e / 16, logit_key(m));
    if constexpr (kPer == 8) m = fmaxf(m, xor_lane_f32<2>(m));
    m = fmaxf(m, xor_lane_f32<4>(m));
    if constexpr (kPer == 4) m = fmaxf(m, xor_lane_f32<8>(m));
    if (P.group_shift == 6 && e % 64 == 0 && e / 64 < P.groups)
      dstore(P.dbg, 5, kDbgSampleWork, P.group_max + row * P.groups + e / 64, logit_key(m));
    if (P.group_shift == 8) {  // of 256: a wave's 64 pieces of 4, or half of its pieces of 8
      if constexpr (kPer == 8) m = fmaxf(m, xor_lane_f32<8>(m));
      m = fmaxf(m, xor_lane_f32<16>(m));
      if constexpr (kPer == 4) m = fmaxf(m, xor_lane_f32<32>(m));
      if (e % 256 == 0 && e / 256 < P.groups)
        dstore(P.dbg, 5, kDbgSampleWork, P.group_max + row * P.groups + e / 256, logit_key(m));
    }
    top = fmaxf(top, m);
  }
  if (mode == kMaximaOnly) return;
  if constexpr (kPer == 8) top = fmaxf(top, xor_lane_f32<8>(top));
  top = fmaxf(top, xor_lane_f32<16>(top));
  top = fmaxf(top, xor_lane_f32<32>(top));
  if (lane == 0) wave_top[tid >> 6] = top;
  if (mode == kMassHistogram)
    for (int i = tid; i < kScanBins; i += kThreads) hist[i] = 0;
  else if (tid < 8)
    eighth[tid] = exp2_f64(tid * (1.0 / 8.0));
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, wave_top[w]);
  const double c8 = 8.0 * S.c;
  const EighthSeries power;
  double sum = 0.0;
  if (mode == kChunkMass) {
    if (top == INFINITY) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += x[p][j] == INFINITY ? 1.0 : 0.0;
    } else if (top > -INFINITY) {
      // 2^(t / 8) as the fraction's power, an eighth's and an exponent; what
      // lies 2^-1000 below the chunk's largest (masked entries among it) adds
      // as much as nothing
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const Eighths e(fmax((static_cast<double>(x[p][j]) - static_cast<double>(top)) * c8, -8000.0));
          const double w = power(e.f) * eighth[e.b & 7];
          sum += __hiloint2double(__double2hiint(w) + ((e.b >> 3) << 20), __double2loint(w));
        }
    }
  } else {
    const double base = rint(static_cast<double>(top) * c8);
    if (grid_fits(base, c8)) {
      const int first = static_cast<int>(base);
      // What lies below the last bin, 2^-64 of the chunk's largest weight, is
      // left out: of 2^20 entries all together less than 2^-44 of the mass.
      // Masked entries and NaN are brought there.
      const float low = static_cast<float>((base - 2.0 * kScanBins) / c8);
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const Eighths e(static_cast<double>(fmaxf(x[p][j], low)) * c8);
          const uint32_t d = static_cast<uint32_t>(first - e.b);
          if (d < kScanBins)
            atomicAdd(reinterpret_cast<unsigned long long*>(&hist[d]),
                      static_cast<unsigned long long>(hist_word(power, e)));
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
    dstore(P.dbg, 5, kDbgSampleWork, P.chunk_max + slot, logit_key(top));
    dstore(P.dbg, 5, kDbgSampleWork, P.chunk_mass + slot, s);
  }
}

template <class T, int kThreads, bool ONCE>
__global__ __launch_bounds__(kThreads) void k_sample_scan(SampleParams P) {
  __shared__ ScanLds<kThreads> lds;
  scan_chunk<T, kThreads, ONCE>(P, P.row0 + blockIdx.x / P.chunks, blockIdx.x % P.chunks, lds);
}

constexpr int kMaxGroups = kSampleMaxGroups;
constexpr int kDistanceBins = 1024;  // of bound_of_kth
constexpr int kFineBits = kRowThreads == 512 ? 9 : 10;
static_assert(1 << kFineBits == kRowThreads, "one of border_entry's bins per thread");
constexpr int kMaxChunks = kSampleMaxChunks;

struct PickLds {
  union {
    struct {
      uint32_t group_max[kMaxGroups];
      union {
        struct {
          uint32_t key[kCandidates];
          int32_t pos[kCandidates];
        } cand;
        struct {
          uint32_t count[kScanBins];
          double mass[kScanBins];
        } half;  // the second half of the block's sums over the chunks
      };
    };
    uint64_t entry[kFlatEntries];  // (key, ~position) of a flat row's border bin
  };
  union {
    uint32_t bins[kDistanceBins];
    uint32_t list[kCandidates];  // groups that reach the bound
    struct {  // finer histogram of the entries among which the border lies
      uint32_t count[kRowThreads];
      uint64_t units[kRowThreads];
    } fine;
  };
  double bin_scale[kScanBins];  // 2^(-d / 8)
  double eighth[8];             // 2^(j / 8)
  double chunk[kMaxChunks];
  uint64_t chunk_units[kMaxChunks];
  int32_t chunk_off[kMaxChunks];
  double wave_f64[6][kRowWaves];
  uint64_t wave_u64[kRowWaves];
  uint32_t wave_u32[6][kRowWaves];
  uint32_t word[10];
  double value;
  uint64_t units;
  uint64_t edge;
  uint32_t few[64];
};

// Exclusive sum of v over the block in thread order; total gets the sum. One
// barrier: `wave` must not have been in use since the last one. Every wave adds
// up the waves' sums in a row of its lanes.
template <class V>
__device__ __forceinline__ V block_scan(V v, V* wave, V& total) {
  static_assert(kRowWaves == 16 || kRowWaves == 8, "within a row of lanes");
  const V incl = wave_scan(v);
  const int lane = threadIdx.x & 63;
  if (lane == 63) wave[threadIdx.x >> 6] = incl;
  __syncthreads();
  V w = wave[lane & (kRowWaves - 1)];
  w += dpp<0x111>(w);
  w += dpp<0x112>(w);
  w += dpp<0x114>(w);
  if constexpr (kRowWaves == 16) w += dpp<0x118>(w);
  total = from_lane(w, kRowWaves - 1);
  const int me = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const V base = me > 0 ? from_lane(w, me - 1) : V(0);
  return base + (incl - v);
}

// Least and largest index of the block at which `hit`, whose lanes' indices
// rise with the lane: one atomic per wave, since those of many lanes on one
// address are carried out one after the other.
__device__ __forceinline__ void put_first(uint32_t* word, bool hit, uint32_t index) {
  const uint64_t b = __ballot(hit);
  if (b && (threadIdx.x & 63) == static_cast<uint32_t>(__ffsll(static_cast<long long>(b)) - 1)) atomicMin(word, index);
}
__device__ __forceinline__ void put_last(uint32_t* word, bool hit, uint32_t index) {
  const uint64_t b = __ballot(hit);
  if (b && (threadIdx.x & 63) == static_cast<uint32_t>(63 - __clzll(static_cast<long long>(b)))) atomicMax(word, index);
}

// One compare-exchange step of a wave's bitonic sort (descending) of 64 R keys,
// lane l holding elements l R .. l R + R - 1.
template <int R, int K, int J>
__device__ __forceinline__ void sort_step(uint32_t (&s)[R]) {
  const int lane = threadIdx.x & 63;
  if constexpr (J < R) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r & J) continue;
      const uint32_t hi = max(s[r], s[r | J]), lo = min(s[r], s[r | J]);
      const bool down = K < R ? (r & K) == 0 : (lane & (K / R)) == 0;
      s[r] = down ? hi : lo;
      s[r | J] = down ? lo : hi;
    }
  } else {
    const bool take_max = ((lane & (J / R)) == 0) == ((lane & (K / R)) == 0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t o = xor_lane<J / R>(s[r]);
      s[r] = take_max ? max(s[r], o) : min(s[r], o);
    }
  }
  if constexpr (J > 1) sort_step<R, K, J / 2>(s);
}

template <int R, int K = 2>
__device__ __forceinline__ void sort_wave(uint32_t (&s)[R]) {
  sort_step<R, K, K / 2>(s);
  if constexpr (K < 64 * R) sort_wave<R, 2 * K>(s);
}

// Border and draw among 64 R entries held by one wave, entry l R + r in lane l
// (keys at or below kMaskedKey: none). whole: the mass that top-p goes by, or
// negative for that of the first k entries. Returns the entry drawn, with its
// weight and that of all kept entries, to every lane. At least one entry must
// be unmasked.
template <int R>
__device__ __forceinline__ int settle_wave(const uint32_t (&key)[R], const RowSettings& S, float m, uint32_t m_key,
                                           double whole, double& w_at, double& kept) {
  const int lane = threadIdx.x & 63;
  double w[R];  // of the entries kept, in their own order
  if (S.k < 64 * R || S.p < 1.0) {
    uint32_t s[R];
    bool falls = true;  // in order already, as a teacher cache's lists are
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = key[r];
      if (r > 0) falls = falls && key[r - 1] >= key[r];
    }
    const uint32_t next = dpp<0x130>(key[0]);  // of the following lane; 0 at the end
    falls = falls && key[R - 1] >= next;
    const bool ordered = __ballot(falls) == ~uint64_t(0);
    if (!ordered) sort_wave<R>(s);
    double mine = 0.0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[r] = static_cast<uint32_t>(lane * R + r) < S.k ? weight_of(s[r], m, m_key, S.c) : 0.0;
      mine += w[r];
    }
    double incl = wave_scan(mine);
    const double target = S.p * (whole < 0.0 ? from_lane(incl, 63) : whole);
    double run = incl - mine;
    uint32_t n_kept = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool keep = static_cast<uint32_t>(lane * R + r) < S.k && s[r] > kMaskedKey &&
                        (S.p >= 1.0 || run < target) && w[r] >= S.q;
      n_kept += __popcll(__ballot(keep));
      run += w[r];
    }
    if (n_kept == 0) n_kept = 1;
    if (ordered) {  // the kept entries are the first ones
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (static_cast<uint32_t>(lane * R + r) >= n_kept) w[r] = 0.0;
    } else {
      const uint32_t last = n_kept - 1;
      uint32_t edge = 0, above = 0, ties = 0;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r == static_cast<int>(last % R)) edge = from_lane(s[r], static_cast<int>(last / R));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        above += __popcll(__ballot(s[r] > edge));
        ties += __popcll(__ballot(s[r] == edge));
      }
      // of the entries equal to the edge, the first this many are kept
      const uint32_t quota = n_kept - above;
      uint32_t before = 0;
      if (quota < ties) {
        uint32_t equal = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) equal += key[r] == edge;
        before = wave_scan(equal) - equal;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool in = key[r] > edge || (key[r] == edge && (quota >= ties || before++ < quota));
        w[r] = in ? weight_of(key[r], m, m_key, S.c) : 0.0;
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[r] = weight_of(key[r], m, m_key, S.c);
      if (w[r] < S.q) w[r] = 0.0;
    }
  }
  double mine = 0.0;
#pragma unroll
  for (int r = 0; r < R; ++r) mine += w[r];
  const double incl = wave_scan(mine);
  kept = from_lane(incl, 63);
  const double goal = S.u * kept;
  double run = incl - mine;
  int hit = R, last = 0;
  double w_hit = 0.0, w_last = 0.0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    run += w[r];
    if (w[r] > 0.0) {
      if (hit == R && run > goal) hit = r, w_hit = w[r];
      last = r, w_last = w[r];
    }
  }
  const uint64_t hits = __ballot(hit < R);
  const uint64_t any = __ballot(w_last > 0.0);
  const int l = hits ? __ffsll(static_cast<long long>(hits)) - 1 : 63 - __clzll(static_cast<long long>(any));
  w_at = hits ? from_lane(w_hit, l) : from_lane(w_last, l);
  return l * R + static_cast<int>(from_lane(static_cast<uint32_t>(hits ? hit : last), l));
}

// Rows of up to 64 R entries, one wave each: latency of one row's chain of
// steps for few rows, vector instructions (about 700 for R = 2) for many. 64
// rows of 100 fp32 logits: 3.5 us; 16384: 9 us, and 20 with top-p, whose border
// takes a sort.
template <class T, int R>
__global__ __launch_bounds__(256) void k_sample_short(SampleParams P, int64_t rows) {
  const int lane = threadIdx.x & 63;
  const int64_t local = blockIdx.x * 4ll + (threadIdx.x >> 6);
  if (local >= rows) return;
  const int64_t row = P.row0 + local;
  const T* x = static_cast<const T*>(P.logits) + row * P.ld;
  uint32_t key[R], m_key = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int at = lane * R + r;
    key[r] = at < P.V ? logit_key(static_cast<float>(dload(P.dbg, 0, kDbgSampleLogits, x + at))) : 0u;
    m_key = max(m_key, key[r]);
  }
  m_key = wave_max_u32(m_key);
  const RowSettings S = row_settings(P, row);
  if (!S.valid || m_key <= kMaskedKey) {
    if (lane == 0) put_none(P, row);
    return;
  }
  double w, total;
  const int at = settle_wave<R>(key, S, key_logit(m_key), m_key, -1.0, w, total);
  if (lane == 0) put_draw(P, row, at, w, total);
}

// Distance of a key from the largest, in bins for bound_of_kth: exact below
// 32, then 32 bins per power of two.
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
__device__ __forceinline__ uint32_t bound_of_kth(PickLds& L, int groups, uint32_t m_key, uint32_t k) {
  const int tid = threadIdx.x;
  constexpr int kPer = kDistanceBins / kRowThreads;
#pragma unroll
  for (int j = 0; j < kPer; ++j) L.bins[tid + j * kRowThreads] = 0;
  if (tid == 0) L.word[0] = kMaskedKey + 1;
  __syncthreads();
  for (int g = tid; g < groups; g += kRowThreads)
    if (L.group_max[g] > kMaskedKey) atomicAdd(&L.bins[distance_bin(m_key - L.group_max[g])], 1u);
  __syncthreads();
  uint32_t mine[kPer], sum = 0, total;
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum += mine[j] = L.bins[tid * kPer + j];
  uint32_t before = block_scan(sum, L.wave_u32[1], total);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (before < k && before + mine[j] >= k) {
      const uint32_t d = distance_bin_end(static_cast<uint32_t>(tid * kPer + j));
      L.word[0] = max(kMaskedKey + 1, d < m_key ? m_key - d : 0u);
    }
    before += mine[j];
  }
  __syncthreads();
  return L.word[0];
}

// The lowest key in (kMaskedKey, m_key] whose bin is at least b; m_key + 1 if
// there is none. Each step tests 64 keys of the range, one per lane.
__device__ __forceinline__ uint32_t first_key_of_bin(double b, double c8, uint32_t m_key) {
  const uint32_t lane = threadIdx.x & 63;
  uint64_t lo = kMaskedKey + 1, hi = static_cast<uint64_t>(m_key) + 1;
  while (lo < hi) {
    const uint64_t step = (hi - lo) / 64 + 1;
    const uint64_t at = lo + lane * step;
    const bool in = at >= hi || rint(static_cast<double>(key_logit(static_cast<uint32_t>(at))) * c8) >= b;
    const uint64_t hit = __ballot(in);
    const int f = hit ? __ffsll(static_cast<long long>(hit)) - 1 : 64;
    if (f < 64) hi = min(hi, lo + f * step);
    if (f > 0) lo = lo + (f - 1) * step + 1;
    else hi = lo;
  }
  return static_cast<uint32_t>(lo);
}

// 2^(t / 8) for t <= 8, by the table L.eighth; 0 below 2^-1000.
__device__ __forceinline__ double power(const PickLds& L, double t) {
  const Eighths e(fmax(t, -8000.0));
  const double w = EighthSeries()(e.f) * L.eighth[e.b & 7];
  const double v = __hiloint2double(__double2hiint(w) + ((e.b >> 3) << 20), __double2loint(w));
  return t < -8000.0 ? 0.0 : v;
}

// The draw within one chunk, from the first position at which base plus the
// kept weights up to it exceeds goal; weight(logit, position) is 0 for what is
// not kept (masked entries among it), kept the sum over the row.
template <class T, class Weight>
__device__ __forceinline__ void draw_in_chunk(const SampleParams& P, int64_t row, const RowView<T>& view, PickLds& L,
                                              int chunk, double base, double goal, double kept, Weight weight) {
  constexpr int kPer = RowView<T>::kPer;
  const int tid = threadIdx.x;
  const int pieces = P.chunk_elems / kPer;
  const int in_row = min(pieces, (view.lead + P.V + kPer - 1) / kPer - chunk * pieces);
  __syncthreads();
  if (tid == 0) L.word[0] = 0xffffffffu, L.word[1] = 0;
  int first_at = -1, last_at = -1;  // this thread's positions past the goal, and of positive weight
  double first_w = 0.0, last_w = 0.0;
  for (int p0 = 0; p0 < in_row; p0 += kRowThreads) {
    float x[kPer];
    double w[kPer], sum = 0.0, total;
    const int piece = chunk * pieces + p0 + tid;
    const int pos = piece * kPer - view.lead;
    const bool live = p0 + tid < in_row;
    if (live) view.logits(P.dbg, piece, x);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      w[j] = live ? weight(x[j], pos + j) : 0.0;
      sum += w[j];
      if (w[j] > 0.0) last_at = pos + j, last_w = w[j];
    }
    __syncthreads();
    double run = base + block_scan(sum, L.wave_f64[5], total);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      run += w[j];
      if (first_at < 0 && w[j] > 0.0 && run > goal) first_at = pos + j, first_w = w[j];
    }
    put_first(&L.word[0], first_at >= 0, static_cast<uint32_t>(first_at));
    put_last(&L.word[1], sum > 0.0, static_cast<uint32_t>(last_at));
    base += total;
    __syncthreads();
    if (L.word[0] != 0xffffffffu) break;
  }
  // if rounding leaves no such position, the last one kept
  const bool found = L.word[0] != 0xffffffffu;
  const int at = static_cast<int>(found ? L.word[0] : L.word[1]);
  if (found ? first_at == at : last_at == at) put_draw(P, row, at, found ? first_w : last_w, kept);
}

// The chunk in which the running sum of L.chunk[0 .. n), n <= 64, exceeds the
// share u of its total (the last one that is not empty if rounding leaves
// none); total, goal = u total, and the sum before the chunk.
__device__ __forceinline__ int find_chunk(const PickLds& L, int n, double u, double& total, double& goal,
                                          double& base) {
  const int lane = threadIdx.x & 63;
  const double w = lane < n ? L.chunk[lane] : 0.0;
  const double incl = wave_scan(w);
  total = from_lane(incl, 63);
  goal = u * total;
  const uint64_t any = __ballot(w > 0.0);
  const uint64_t hit = __ballot(w > 0.0 && incl > goal);
  const int at = hit ? __ffsll(static_cast<long long>(hit)) - 1 : 63 - __clzll(static_cast<long long>(any));
  base = from_lane(incl - w, at);
  return at;
}

// What the mass histograms say of a row.
struct RowHistogram {
  double c8, base;   // the grid, and the bin of the row's largest logit
  double whole;       // the row's mass relative to 2^(base / 8)
  uint32_t border;    // the bin (from the top) in which the mass reaches target, or the count top-k
  uint32_t in_border, above;  // entries in it and above it
  double mass_above;
  double target;
};

// Adds up a row's histograms and finds the border bin; false where it lies
// below the bins.
__device__ __forceinline__ bool row_histogram(const SampleParams& P, int64_t slot, const RowSettings& S, float m,
                                              PickLds& L, RowHistogram& H) {
  const int tid = threadIdx.x;
  H.c8 = 8.0 * S.c;
  H.base = rint(static_cast<double>(m) * H.c8);
  if (!grid_fits(H.base, H.c8)) return false;
  if (tid < P.chunks) {
    const uint32_t ck = dload(P.dbg, 5, kDbgSampleWork, P.chunk_max + slot + tid);
    // chunk bin i is row bin i + off; a masked chunk's are all empty
    const double off = ck > kMaskedKey ? H.base - rint(static_cast<double>(key_logit(ck)) * H.c8) : 1e6;
    L.chunk_off[tid] = static_cast<int>(fmin(off, 1e6));
  }
  if (tid < kScanBins) L.bin_scale[tid] = power(L, -tid);
  if (tid == 0) L.word[2] = 0xffffffffu;
  __syncthreads();
  // the block's parts of kScanBins threads take turns at the chunks
  const int bin = tid % kScanBins;
  uint32_t count = 0;
  double mass = 0.0;
  constexpr int kBatch = 8;  // words read before any is used
  for (int c0 = tid / kScanBins; c0 < P.chunks; c0 += kBatch * (kRowThreads / kScanBins)) {
    uint64_t w[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int ch = c0 + b * (kRowThreads / kScanBins);
      w[b] = 0;
      if (ch < P.chunks) {
        const int off = L.chunk_off[ch];
        if (off <= bin) w[b] = dload(P.dbg, 5, kDbgSampleWork, P.chunk_hist + (slot + ch) * kScanBins + bin - off);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) count += hist_count(w[b]), mass += units_mass(hist_units(w[b]));
  }
  if constexpr (kRowThreads > kScanBins) {
    if (tid >= kScanBins) L.half.count[bin] = count, L.half.mass[bin] = mass;
    __syncthreads();
    if (tid < kScanBins) count += L.half.count[bin], mass += L.half.mass[bin];
    else count = 0, mass = 0.0;
  }
  const double scaled = tid < kScanBins ? mass * L.bin_scale[bin] : 0.0;
  uint32_t counted;
  const double above = block_scan(scaled, L.wave_f64[0], H.whole);
  const uint32_t count_above = block_scan(count, L.wave_u32[2], counted);
  H.target = S.p * H.whole;
  const bool here = S.k < static_cast<uint32_t>(P.V) ? count_above < S.k && count_above + count >= S.k
                                                     : above < H.target && above + scaled >= H.target;
  put_first(&L.word[2], count > 0 && here, static_cast<uint32_t>(tid));
  __syncthreads();
  H.border = L.word[2];
  if (H.border == 0xffffffffu) return false;
  if (static_cast<uint32_t>(tid) == H.border) L.word[3] = count, L.word[4] = count_above, L.value = above;
  __syncthreads();
  H.in_border = L.word[3];
  H.above = L.word[4];
  H.mass_above = L.value;
  return true;
}

// Keys of 16-bit logits differ in their upper bits alone: a bin of 2^GRAIN keys,
// aligned to that, holds one of them.
template <class T>
constexpr int kGrain = std::is_same<T, __bf16>::value ? 16 : std::is_same<T, _Float16>::value ? 13 : 0;

// The last entry kept of a list in LDS: the last, in the order of (key
// descending, position ascending), before which the entries of keys in [lo,
// hi) amount to less than `target`: their number, or the units of their
// weights. entry(i) = (key, ~position), 0 <= i < n, so that larger values come
// first; at least one entry has a key in [lo, hi) and target > 0. The keys are
// counted into a bin per thread, then those of the bin at which the target is reached
// again, until that bin holds at most 64 entries, which one wave compares, or
// entries of one key, of which the last one's position is looked for among as
// many bins of positions. Returns the entry to every thread.
template <int GRAIN, class Entry, class Units>
__device__ __forceinline__ uint64_t border_entry(PickLds& L, int V, int n, uint32_t lo, uint64_t hi, bool by_units,
                                                 uint64_t target, Entry entry, Units units) {
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  uint64_t above = 0;
  int count;
  lo &= ~((1u << GRAIN) - 1);
  for (;;) {
    const uint32_t span = static_cast<uint32_t>(hi - lo - 1);
    const int shift = max(GRAIN, 32 - kFineBits - __clz(static_cast<int>(span | 1)));
    __syncthreads();
    L.fine.count[tid] = 0;
    L.fine.units[tid] = 0;
    if (tid == 0) L.word[5] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kRowThreads) {
      const uint32_t key = static_cast<uint32_t>(entry(i) >> 32);
      if (key < lo || key >= hi) continue;
      // 16-bit logits come in few values: lanes of the first lane's key are counted at once
      const uint32_t lead = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(key)));
      const uint64_t same = __ballot(key == lead);
      const uint32_t times = key != lead ? 1u : lane == __ffsll(static_cast<long long>(same)) - 1 ? __popcll(same) : 0u;
      if (times == 0) continue;
      atomicAdd(&L.fine.count[(key - lo) >> shift], times);
      if (by_units)
        atomicAdd(reinterpret_cast<unsigned long long*>(&L.fine.units[(key - lo) >> shift]),
                  static_cast<unsigned long long>(units(key) * times));
    }
    __syncthreads();
    const int bin = kRowThreads - 1 - tid;
    const uint32_t here = L.fine.count[bin];
    uint64_t sum;
    const uint64_t before = above + block_scan(by_units ? L.fine.units[bin] : uint64_t(here), L.wave_u64, sum);
    put_last(&L.word[5], here > 0 && before < target, static_cast<uint32_t>(tid));
    __syncthreads();
    const int at = static_cast<int>(L.word[5]);
    if (tid == at) L.word[6] = here, L.units = before;
    __syncthreads();
    count = static_cast<int>(L.word[6]);
    above = L.units;
    lo += static_cast<uint32_t>(kRowThreads - 1 - at) << shift;
    hi = min(hi, static_cast<uint64_t>(lo) + (uint64_t(1) << shift));
    if (count <= 64 || shift == GRAIN) break;
  }
  L.few[lane] = 0;
  if (tid == 0) L.word[7] = 0;
  __syncthreads();
  if (count <= 64) {
    for (int i = tid; i < n; i += kRowThreads) {
      const uint32_t key = static_cast<uint32_t>(entry(i) >> 32);
      if (key >= lo && key < hi) L.few[atomicAdd(&L.word[7], 1u)] = static_cast<uint32_t>(i);
    }
    __syncthreads();
    if (tid < 64) {
      const uint64_t mine = lane < count ? entry(static_cast<int>(L.few[lane])) : 0;
      const uint64_t w = by_units ? units(static_cast<uint32_t>(mine >> 32)) : 1;
      uint64_t before = above;
      for (int i = 0; i < count; ++i)
        if (from_lane(mine, i) > mine) before += from_lane(w, i);
      uint64_t last = ~uint64_t(0);  // of those kept; the first one is, above < target
      for (uint64_t left = __ballot(lane < count && before < target); left; left &= left - 1)
        last = min(last, from_lane(mine, __ffsll(static_cast<long long>(left)) - 1));
      if (lane == 0) L.edge = last;
    }
  } else {
    // the key whose bin it is: positive logits' lower bits are 0, negative ones' 1
    if (!(lo & 0x80000000u)) lo |= (1u << GRAIN) - 1;
    const uint64_t each = by_units ? max(units(lo), uint64_t(1)) : 1;
    const uint64_t want = (target - above + each - 1) / each;  // >= 1
    const uint32_t quota = static_cast<uint32_t>(min(want, static_cast<uint64_t>(count)));
    int pos_shift = 0;
    while ((V - 1) >> pos_shift >= kRowThreads) ++pos_shift;
    L.bins[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t e = entry(i);
      if (static_cast<uint32_t>(e >> 32) == lo) atomicAdd(&L.bins[~static_cast<uint32_t>(e) >> pos_shift], 1u);
    }
    __syncthreads();
    const uint32_t here = L.bins[tid];
    uint32_t all;
    const uint32_t before = block_scan(here, L.wave_u32[3], all);
    if (before < quota && before + here >= quota) L.word[8] = static_cast<uint32_t>(tid), L.word[9] = quota - before;
    __syncthreads();
    const uint32_t pos_bin = L.word[8];
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t e = entry(i);
      const uint32_t pos = ~static_cast<uint32_t>(e);
      if (static_cast<uint32_t>(e >> 32) == lo && pos >> pos_shift == pos_bin) {
        const uint32_t bit = pos & ((1u << pos_shift) - 1);  // of at most 64 * 32
        atomicOr(&L.few[bit >> 5], 1u << (bit & 31));
      }
    }
    __syncthreads();
    if (tid < 64) {
      uint32_t bits = L.few[lane];
      const uint32_t c = static_cast<uint32_t>(__popc(bits));
      const uint32_t before_c = wave_scan(c) - c;
      uint32_t nth = L.word[9];
      if (before_c < nth && before_c + c >= nth) {
        while (--nth > before_c) bits &= bits - 1;
        const uint32_t pos = (pos_bin << pos_shift) + static_cast<uint32_t>(lane * 32 + __ffs(static_cast<int>(bits)) - 1);
        L.edge = (static_cast<uint64_t>(lo) << 32) | ~pos;
      }
    }
  }
  __syncthreads();
  return L.edge;
}

// Elements of a 16-bit type in [x_lo, x_hi), two at a time, where the range
// does not reach zero: their bits are consecutive there, the magnitudes rising.
template <class T>
struct Range16 {
  bool one_sign;
  uint32_t first, count;  // twice in a word
  // the least bits of a magnitude that is at least y, or larger than y
  static __device__ __forceinline__ uint32_t least(float y, bool larger) {
    if constexpr (sizeof(T) == 2) {
      const T t = static_cast<T>(y);  // the nearest: its neighbour below is too small
      const float v = static_cast<float>(t);
      return __builtin_bit_cast(uint16_t, t) + (v < y || (larger && v == y) ? 1u : 0u);
    }
    return 0;
  }
  __device__ __forceinline__ Range16(float x_lo, float x_hi) {
    one_sign = x_lo > 0.0f || x_hi < 0.0f;
    const bool minus = x_hi < 0.0f;
    const uint32_t a = minus ? least(-x_hi, true) : least(x_lo, false);
    const uint32_t b = minus ? least(-x_lo, true) : least(x_hi, false);
    first = (a | (minus ? 0x8000u : 0u)) * 0x10001u;
    count = (b - a) * 0x10001u;
  }
  // 1 in each half of the word whose element is in the range
  __device__ __forceinline__ uint32_t inside(uint32_t word) const {
    const u16x2 from = __builtin_bit_cast(u16x2, word) - __builtin_bit_cast(u16x2, first);
    const u16x2 left = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, count), from);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(left, u16x2{1, 1}));
  }
};

// A row of which more entries are kept than the workgroup holds: the bins
// above the border are kept whole, and only the border bin's entries are
// gathered (one read of the row, two where they are more than 6144) and
// settled. false where thousands of them are equal.
template <class T>
__device__ __forceinline__ bool pick_flat_row(const SampleParams& P, int64_t row, const RowSettings& S,
                                              const RowView<T>& view, uint32_t m_key, PickLds& L,
                                              const RowHistogram& H) {
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int V = P.V;
  const int64_t slot = row * P.chunks;
  const bool by_count = S.k < static_cast<uint32_t>(V);
  if (by_count && (S.p < 1.0 || S.q > 0.0)) return false;
  const double edge_bin = H.base - H.border;
  if (wave < 2) {
    const uint32_t key = first_key_of_bin(edge_bin + wave, H.c8, m_key);
    if (lane == 0) L.word[wave] = key;
  }
  if (tid < P.chunks) L.chunk_units[tid] = 0;
  if (tid == 0) L.word[2] = 0;
  __syncthreads();
  const uint32_t bin_end = L.word[1];
  uint32_t k_lo = L.word[0], k_hi = bin_end;  // the keys among which the border lies
  auto units = [&](uint32_t key) {
    return hist_units(hist_word(EighthSeries(), Eighths(static_cast<double>(key_logit(key)) * H.c8)));
  };
  const double scale = L.bin_scale[H.border] * (1.0 / (uint64_t(1) << kHistShift));  // of the border bin's units
  const double want = ceil((H.target - H.mass_above) / scale);
  uint64_t target = by_count ? S.k - H.above : want < 1.0 ? 1 : static_cast<uint64_t>(want);
  constexpr int kPer = RowView<T>::kPer;
  const int pieces = (view.lead + V + kPer - 1) / kPer;
  constexpr int kBatch = 4;  // pieces read before any is looked at
  int n = static_cast<int>(H.in_border);
  if (n > kFlatEntries) {
    // one more read of the row: the bin's entries counted into finer bins
    const int shift = max(0, 32 - kFineBits - __clz(static_cast<int>((k_hi - k_lo - 1) | 1)));
    const float x_lo = key_logit(k_lo), x_hi = key_logit(k_hi);
    L.fine.count[tid] = 0;
    L.fine.units[tid] = 0;
    if (tid == 0) L.word[5] = 0;
    __syncthreads();
    for (int p0 = 0; p0 < pieces; p0 += kBatch * kRowThreads) {
      u32x4 held[kBatch];
      view.template batch<kBatch>(P.dbg, p0, kRowThreads, held);
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float x = view.logit(held[b], j);
          if (x >= x_lo && x < x_hi) {
            const uint32_t key = logit_key(x);
            atomicAdd(&L.fine.count[(key - k_lo) >> shift], 1u);
            atomicAdd(reinterpret_cast<unsigned long long*>(&L.fine.units[(key - k_lo) >> shift]),
                      static_cast<unsigned long long>(units(key)));
          }
        }
    }
    __syncthreads();
    const uint32_t here = L.fine.count[kRowThreads - 1 - tid];
    uint64_t sum;
    const uint64_t before =
        block_scan(by_count ? uint64_t(here) : L.fine.units[kRowThreads - 1 - tid], L.wave_u64, sum);
    put_last(&L.word[5], here > 0 && before < target, static_cast<uint32_t>(tid));
    __syncthreads();
    const int at = static_cast<int>(L.word[5]);
    if (tid == at) L.word[6] = here, L.units = before;
    __syncthreads();
    n = static_cast<int>(L.word[6]);
    target -= L.units;
    k_lo += static_cast<uint32_t>(kRowThreads - 1 - at) << shift;
    k_hi = static_cast<uint32_t>(min(static_cast<uint64_t>(k_hi), static_cast<uint64_t>(k_lo) + (uint64_t(1) << shift)));
    if (n > kFlatEntries) return false;  // thousands of equal entries
    __syncthreads();
  }
  const float x_lo = key_logit(k_lo), x_hi = key_logit(k_hi), x_end = key_logit(bin_end);
  const Range16<T> range(x_lo, x_hi);
  for (int p0 = 0; p0 < pieces; p0 += kBatch * kRowThreads) {  // the same for all lanes: they vote below
    const int i0 = p0 + tid;
    u32x4 held[kBatch];
    view.template batch<kBatch>(P.dbg, p0, kRowThreads, held);
    if (x_hi < x_end) {  // the bin's entries above the finer one are kept: their chunk's mass
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        uint64_t kept = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float x = view.logit(held[b], j);
          if (x >= x_hi && x < x_end) kept += units(logit_key(x));
        }
        if (__ballot(kept != 0) != 0) {  // a wave's pieces lie in one chunk
          const uint64_t all = from_lane(wave_scan(kept), 63);
          if (lane == 0)
            atomicAdd(reinterpret_cast<unsigned long long*>(
                          &L.chunk_units[(i0 + b * kRowThreads) * kPer / P.chunk_elems]),
                      static_cast<unsigned long long>(all));
        }
      }
    }
    // bit b kPer + j: element j of piece b; for 16-bit types bit 4 b + i: element 2 i, 16 more: 2 i + 1
    uint32_t hits = 0;
    if (sizeof(T) == 2 && range.one_sign) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) hits |= range.inside(held[b][i]) << (b * 4 + i);
    } else {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float x = view.logit(held[b], j);
          const int bit = sizeof(T) == 2 ? b * 4 + j / 2 + j % 2 * 16 : b * kPer + j;
          hits |= (x >= x_lo && x < x_hi ? 1u : 0u) << bit;
        }
    }
    const uint32_t mine = static_cast<uint32_t>(__popc(hits));
    const uint32_t incl = wave_scan(mine);
    uint32_t at = 0;
    if (lane == 63) at = atomicAdd(&L.word[2], incl);
    at = from_lane(at, 63) + incl - mine;
    for (; hits; hits &= hits - 1, ++at) {
      const int bit = __ffs(static_cast<int>(hits)) - 1;
      const int b = bit / 4 % 4, j = sizeof(T) == 2 ? bit % 4 * 2 + bit / 16 : bit % 4;
      if (at < kFlatEntries) L.entry[at] = static_cast<uint32_t>((i0 + b * kRowThreads) * kPer + j - view.lead);
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += kRowThreads) {
    const uint32_t pos = static_cast<uint32_t>(L.entry[i]);
    L.entry[i] = (static_cast<uint64_t>(view.element(P.dbg, static_cast<int>(pos) + view.lead)) << 32) | ~pos;
  }
  const uint64_t edge = border_entry<kGrain<T>>(L, V, n, k_lo, k_hi, !by_count, target, [&](int i) { return L.entry[i]; }, units);
  const uint32_t edge_key = static_cast<uint32_t>(edge >> 32);
  const int edge_pos = static_cast<int>(~static_cast<uint32_t>(edge));
  // each chunk's kept mass: its bins above the border, and its kept entries of the border bin
  for (int i = tid; i < n; i += kRowThreads) {
    const uint64_t e = L.entry[i];
    if (e >= edge) {
      const int at = static_cast<int>(~static_cast<uint32_t>(e)) + view.lead;
      atomicAdd(reinterpret_cast<unsigned long long*>(&L.chunk_units[at / P.chunk_elems]),
                static_cast<unsigned long long>(units(static_cast<uint32_t>(e >> 32))));
    }
  }
  __syncthreads();
  const int border = static_cast<int>(H.border);
  for (int ch = wave; ch < P.chunks; ch += kRowWaves) {
    const int off = L.chunk_off[ch];
    double s = 0.0;
    uint64_t w[kScanBins / 64];  // read before any is used, and in any case: no branch to wait in
#pragma unroll
    for (int i = 0; i < kScanBins / 64; ++i)
      w[i] = dload(P.dbg, 5, kDbgSampleWork, P.chunk_hist + (slot + ch) * kScanBins + i * 64 + lane);
#pragma unroll
    for (int i = 0; i < kScanBins / 64; ++i) {
      const int d = i * 64 + lane;
      if (d < border - off) s += units_mass(hist_units(w[i])) * L.bin_scale[off + d];
    }
    s = wave_sum_f64(s);
    if (lane == 0) L.chunk[ch] = s + static_cast<double>(L.chunk_units[ch]) * scale;
  }
  __syncthreads();
  double kept, goal, before;
  const int chunk = find_chunk(L, P.chunks, S.u, kept, goal, before);
  const float edge_x = key_logit(edge_key);
  draw_in_chunk(P, row, view, L, chunk, before, goal, kept, [&](float x, int pos) {
    return x > edge_x || (x == edge_x && pos <= edge_pos) ? power(L, static_cast<double>(x) * H.c8 - H.base) : 0.0;
  });
  return true;
}

template <int R>
__device__ __forceinline__ void settle_candidates(const SampleParams& P, int64_t row, const RowSettings& S, float m,
                                                  uint32_t m_key, const PickLds& L, int n, double whole) {
  const int lane = threadIdx.x & 63;
  uint32_t key[R];
#pragma unroll
  for (int r = 0; r < R; ++r) key[r] = lane * R + r < n ? L.cand.key[lane * R + r] : 0u;
  double w, total;
  const int at = settle_wave<R>(key, S, m, m_key, whole, w, total);
  if (lane == 0) put_draw(P, row, L.cand.pos[at], w, total);
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
  const RowMode mode = row_mode(S, P);
  const float m = key_logit(m_key);
  const int64_t slot = row * P.chunks;
  const bool all = S.k >= static_cast<uint32_t>(V);  // top-k is off

  double whole = -1.0;  // the mass that top-p goes by, relative to m; negative: that of the first k entries
  if (mode == kChunkMass) {
    if (tid < P.chunks) {
      const uint32_t ck = dload(P.dbg, 5, kDbgSampleWork, P.chunk_max + slot + tid);
      const double cm = dload(P.dbg, 5, kDbgSampleWork, P.chunk_mass + slot + tid);
      L.chunk[tid] = ck > kMaskedKey ? cm * weight_of(ck, m, m_key, S.c) : 0.0;
    }
    __syncthreads();
    double goal, base;
    const int chunk = find_chunk(L, P.chunks, S.u, whole, goal, base);
    if (S.p >= 1.0) {  // no filter: a chunk, then a position in it
      draw_in_chunk(P, row, view, L, chunk, base, goal, whole, [&](float x, int) {
        const double d = x == m ? 0.0 : static_cast<double>(x) - static_cast<double>(m);  // m may be infinite
        return x > -INFINITY ? power(L, d * (8.0 * S.c)) : 0.0;
      });
      return true;
    }
  }

  // a key that every kept entry reaches
  uint32_t bound = kMaskedKey + 1;
  if (!all && mode == kMaximaOnly) bound = S.k == 1 ? m_key : bound_of_kth(L, P.groups, m_key, S.k);
  if (S.q > 0.0 && isfinite(m) && (S.p >= 1.0 || whole >= 0.0)) {
    // w >= q: x >= m + log2(q) / c, taken lower by more than its rounding
    // (without the row's mass, top-p needs that of all the entries here: no bound from q then)
    const double lo = static_cast<double>(m) + log2(S.q) / S.c;
    const float low = static_cast<float>(lo - 1e-6 * fabs(lo) - 1e-30);
    bound = max(bound, logit_key(low));
  }
  if (mode == kMassHistogram) {
    RowHistogram H;
    if (!row_histogram(P, slot, S, m, L, H)) return false;
    const bool wide = H.above + H.in_border > (all ? kFlatRow : kCandidates);
    if (wide && (all || S.p < 1.0 || S.q <= 0.0)) return pick_flat_row(P, row, S, view, m_key, L, H);
    if (all) whole = H.whole * exp2_f64((H.base - static_cast<double>(m) * H.c8) * (1.0 / 8.0));
    bound = max(bound, first_key_of_bin(H.base - H.border, H.c8, m_key));
  }

  // The groups that reach the bound, in order, and their entries that do: the
  // candidates, in order of position.
  uint32_t n_list;
  {
    const int per = (P.groups + kRowThreads - 1) / kRowThreads;
    const int g0 = min(tid * per, P.groups), g1 = min(g0 + per, P.groups);
    uint32_t mine = 0;
    for (int g = g0; g < g1; ++g) mine += L.group_max[g] >= bound;
    uint32_t at = block_scan(mine, L.wave_u32[4], n_list);
    if (n_list > kCandidates) return false;
    for (int g = g0; g < g1; ++g)
      if (L.group_max[g] >= bound) L.list[at++] = static_cast<uint32_t>(g);
  }
  __syncthreads();
  // Each thread reads a run of kRun pieces of the listed groups and appends the
  // entries that reach the bound behind those of the threads before it.
  constexpr int kPer = RowView<T>::kPer;
  constexpr int kRun = 4;
  const float bound_x = key_logit(bound);
  const int shift = P.group_shift - (kPer == 8 ? 3 : 2);  // pieces of a group
  const int pieces = static_cast<int>(n_list) << shift;
  uint32_t n_cand = 0;
  for (int p0 = 0, turn = 0; p0 < pieces; p0 += kRun * kRowThreads, turn ^= 1) {
    u32x4 held[kRun];
    int piece[kRun];
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      const int i = p0 + tid * kRun + r;
      piece[r] = i < pieces ? static_cast<int>(L.list[i >> shift] << shift) + (i & ((1 << shift) - 1)) : -1;
    }
#pragma unroll
    for (int r = 0; r < kRun; ++r) held[r] = view.whole(P.dbg, piece[r]);
    uint32_t hits[kRun], mine = 0, sum;
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      if (!view.is_whole(piece[r]) && piece[r] >= 0) held[r] = view.raw(P.dbg, piece[r]);  // the row's first and last
      hits[r] = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) hits[r] |= (view.logit(held[r], j) >= bound_x ? 1u : 0u) << j;
      if (piece[r] < 0) hits[r] = 0;
      mine += static_cast<uint32_t>(__popc(hits[r]));
    }
    uint32_t at = n_cand + block_scan(mine, L.wave_u32[turn ? 5 : 3], sum);
    if (mine > 0) {
#pragma unroll
      for (int r = 0; r < kRun; ++r)
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (((hits[r] >> j) & 1u) && at < kCandidates) {
            L.cand.key[at] = logit_key(view.logit(held[r], j));
            L.cand.pos[at++] = piece[r] * kPer + j - view.lead;
          }
    }
    n_cand += sum;
    if (n_cand > kCandidates) return false;
  }
  __syncthreads();
  const int n = static_cast<int>(n_cand);
  if (n <= kWaveCandidates) {  // one wave settles them without a barrier
    if (wave == 0) settle_candidates<kWaveCandidates / 64>(P, row, S, m, m_key, L, n, whole);
    return true;
  }
  auto weight = [&](uint32_t key) {
    const float x = key_logit(key);
    return x == m ? 1.0 : power(L, (static_cast<double>(x) - static_cast<double>(m)) * (8.0 * S.c));
  };
  constexpr double kUnit = static_cast<double>(uint64_t(1) << 46);  // 4096 weights of at most 1 stay below 2^59
  auto units = [&](uint32_t key) { return static_cast<uint64_t>(weight(key) * kUnit + 0.5); };
  auto entry = [&](int i) {
    return (static_cast<uint64_t>(L.cand.key[i]) << 32) | ~static_cast<uint32_t>(L.cand.pos[i]);
  };
  uint64_t edge = 0;
  if (S.k < static_cast<uint32_t>(n))
    edge = border_entry<kGrain<T>>(L, V, n, bound, uint64_t(m_key) + 1, false, S.k, entry, units);
  if (S.p < 1.0) {
    if (whole < 0.0) {
      double s = 0.0;
      for (int i = tid; i < n; i += kRowThreads)
        if (entry(i) >= edge) s += weight(L.cand.key[i]);
      block_scan(s, L.wave_f64[2], whole);
    }
    const uint64_t target = max(static_cast<uint64_t>(ceil(S.p * whole * kUnit)), uint64_t(1));
    edge = max(edge, border_entry<kGrain<T>>(L, V, n, bound, uint64_t(m_key) + 1, true, target, entry, units));
  }
  // the draw: thread t holds candidates t * per .. in order of position
  constexpr int kPerThread = kCandidates / kRowThreads;
  const int per = (n + kRowThreads - 1) / kRowThreads;
  double w[kPerThread], sum = 0.0, total;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = tid * per + j;
    w[j] = 0.0;
    if (j < per && i < n && entry(i) >= edge) {
      w[j] = weight(L.cand.key[i]);
      if (w[j] < S.q) w[j] = 0.0;
    }
    sum += w[j];
  }
  if (tid == 0) L.word[2] = 0xffffffffu, L.word[3] = 0;
  __syncthreads();
  double run = block_scan(sum, L.wave_f64[4], total);
  const double goal = S.u * total;
  int hit = -1, last = -1;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    run += w[j];
    if (w[j] > 0.0) {
      if (hit < 0 && run > goal) hit = tid * per + j;
      last = tid * per + j;
    }
  }
  put_first(&L.word[2], hit >= 0, static_cast<uint32_t>(hit));
  put_last(&L.word[3], last >= 0, static_cast<uint32_t>(last));
  __syncthreads();
  if (tid == 0) {
    const uint32_t i = L.word[2] != 0xffffffffu ? L.word[2] : L.word[3];
    put_draw(P, row, L.cand.pos[i], weight(L.cand.key[i]), total);
  }
  return true;
}

union RowLds {
  ScanLds<kRowThreads> scan;
  PickLds pick;
  ExactLds exact;
};

template <class T>
__device__ __forceinline__ void pick_or_exact(const SampleParams& P, int64_t row, int shift, RowLds& lds) {
  PickLds& L = lds.pick;
  const int tid = threadIdx.x;
  uint32_t m_key = 0;
  for (int g = tid; g < P.groups; g += kRowThreads) {
    const uint32_t v = dload(P.dbg, 5, kDbgSampleWork, P.group_max + row * P.groups + g);
    L.group_max[g] = v;
    m_key = max(m_key, v);
  }
  const RowSettings S = row_settings(P, row);
  const RowView<T> view(P, row);
  m_key = wave_max_u32(m_key);
  if ((tid & 63) == 0) L.wave_u32[0][tid >> 6] = m_key;
  if (tid < 8) L.eighth[tid] = exp2_f64(tid * (1.0 / 8.0));
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowWaves; ++w) m_key = max(m_key, L.wave_u32[0][w]);
  if (!S.valid || m_key <= kMaskedKey) {
    if (tid == 0) put_none(P, row);
    return;
  }
  if (pick_row<T>(P, row, S, view, m_key, L)) return;
  __syncthreads();
  sample_row_exact<T>(P, row, S, m_key, shift, lds.exact);
}

// One workgroup per row, after k_sample_scan. Latency bound: a chain of short
// steps over LDS, with one dependent read of the groups that reach the bound (9
// us for one row and top-k 50). Where top-p keeps thousands of entries, one CU's
// vector instructions bound it: of the 27 us for a row of 128256 bf16 logits, 3.4
// add up the histograms, 8 gather the border bin, 4 to 6 find the border in it,
// 5 draw.
// Up to one row per CU, a workgroup's waves have all of its registers (87);
// with more rows two workgroups share it (64 registers, some spilled): 512 rows
// of 201088 fp32 logits, 24 instead of 32 us; 64 rows of 128256 bf16 logits 32
// instead of 30 us.
template <class T, int WAVES>
__global__ __launch_bounds__(kRowThreads, WAVES) void k_sample_pick(SampleParams P, int shift) {
  __shared__ RowLds lds;
  pick_or_exact<T>(P, P.row0 + blockIdx.x, shift, lds);
}

// Scan and pick of a row of one chunk, up to one row per CU: what the scan
// leaves is read by the workgroup that wrote it. Launch bound.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_sample_row(SampleParams P, int shift) {
  __shared__ RowLds lds;
  const int64_t row = P.row0 + blockIdx.x;
  scan_chunk<T, kRowThreads, false>(P, row, 0, lds.scan);
  __syncthreads();
  pick_or_exact<T>(P, row, shift, lds);
}

// Rows longer than the scan takes: the largest key, then sample_row_exact, all
// of it by one CU per row (300001 fp32 logits: 0.35 ms without filters, 1.6 ms
// with top-p).
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
  const int regs = static_cast<int>(ceil_div(p.V, 64));  // a short row's entries per lane
  const int64_t rows_max = std::max<int64_t>(1, (int64_t(1) << 21) / per_row);
  const bool once = p.N * p.V * static_cast<int64_t>(sizeof(T)) > kLastLevelBytes;
  for (int64_t r = 0; r < p.N; r += rows_max) {
    const int64_t rows = std::min(p.N - r, rows_max);
    const double bytes = static_cast<double>(rows) * p.V * sizeof(T);
    P.row0 = r;
    if (p.route == kSampleShort) {
      auto* k = regs <= 1   ? k_sample_short<T, 1>
                : regs <= 2 ? k_sample_short<T, 2>
                : regs <= 4 ? k_sample_short<T, 4>
                : regs <= 8 ? k_sample_short<T, 8>
                            : k_sample_short<T, 16>;
      TraceScope ts(st, "sample_short", 0.0, bytes);
      hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(ceil_div(rows, 4))), dim3(256), 0, st, P, rows);
      continue;
    }
    if (p.route == kSampleRow) {
      TraceScope ts(st, "sample_row", 0.0, bytes);
      hipLaunchKernelGGL(k_sample_row<T>, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, st, P, shift);
      continue;
    }
    if (p.route == kSampleLong) {
      TraceScope ts(st, "sample_long", 0.0, bytes);
      hipLaunchKernelGGL(k_sample_long<T>, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, st, P, shift);
      continue;
    }
    {
      TraceScope ts(st, "sample_scan", 0.0, bytes);
      const dim3 grid(static_cast<unsigned>(rows * p.chunks));
      const int threads = static_cast<int>(p.chunk_elems / kScanElems);
      auto* const scan = threads == 256   ? once ? k_sample_scan<T, 256, true> : k_sample_scan<T, 256, false>
                         : threads == 512 ? once ? k_sample_scan<T, 512, true> : k_sample_scan<T, 512, false>
                                          : once ? k_sample_scan<T, 1024, true> : k_sample_scan<T, 1024, false>;
      hipLaunchKernelGGL(scan, grid, dim3(static_cast<unsigned>(threads)), 0, st, P);
    }
    TraceScope ts(st, "sample_pick", 0.0, 4.0 * rows * p.groups);
    auto* const pick = rows > kTargetBlocks ? k_sample_pick<T, 8> : k_sample_pick<T, 4>;
    hipLaunchKernelGGL(pick, dim3(static_cast<unsigned>(rows)), dim3(kRowThreads), 0, st, P, shift);
  }
}

hipError_t launch_sample(const SamplePlan& p, const SampleArgs& a, hipStream_t st) {
  SampleParams P;
  P.logits = a.logits, P.ld = p.ld;
  P.ids = a.ids, P.ld_ids = p.ld_ids;
  P.u = a.u, P.set = a.params;
  P.c = 1.4426950408889634074 / static_cast<double>(a.params.temperature);  // not used where T = 0
  P.token = a.token, P.logprob = a.logprob;
  P.V = static_cast<int32_t>(p.V);
  P.groups = static_cast<int32_t>(p.groups);
  P.group_shift = p.group_shift;
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
                            {a.ws, p.bytes}});
  // V weights of at most 2^shift each stay below 2^63
  int shift = 46;
  while ((p.V >> (62 - shift)) > 0) --shift;
  if (p.type == FKL_F32) launch_sample_of<float>(p, P, shift, st);
  else if (p.type == FKL_BF16) launch_sample_of<__bf16>(p, P, shift, st);
  else launch_sample_of<_Float16>(p, P, shift, st);
  return hipGetLastError();
}

}  // namespace fkl
