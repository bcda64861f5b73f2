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

constexpr int kDigits = 256;

// One workgroup per row, any row: the border by radix selection over the row's
// keys, eight bits at a time, first by count (top-k), then by mass (top-p),
// and the draw by find_position. The masses of the selection are integers in
// units of 2^-shift, whose sum does not depend on its order.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_sample_row(SampleParams P, int shift) {
  __shared__ double shared[kRowWaves + 1];
  __shared__ uint64_t mass[kDigits];
  __shared__ uint32_t count[kDigits];
  __shared__ uint32_t pick[2];
  __shared__ uint64_t pick_mass[2];
  const int tid = threadIdx.x;
  const int64_t row = P.row0 + blockIdx.x;
  const RowSettings S = row_settings(P, row);
  const T* x = static_cast<const T*>(P.logits) + row * P.ld;
  auto key_at = [&](int i) { return logit_key(static_cast<float>(dload(P.dbg, 0, kDbgSampleLogits, x + i))); };
  const int V = P.V;

  uint32_t m_key = 0;
  for (int i = tid; i < V; i += kRowThreads) m_key = max(m_key, key_at(i));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m_key = max(m_key, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m_key), o, 64)));
  if ((tid & 63) == 0) count[tid >> 6] = m_key;
  __syncthreads();
  for (int w = 0; w < kRowWaves; ++w) m_key = max(m_key, count[w]);
  __syncthreads();
  if (!S.valid || m_key <= kMaskedKey) {
    if (tid == 0) {
      dstore(P.dbg, 3, kDbgSampleOut, P.token + row, int32_t(-1));
      if (P.logprob) dstore(P.dbg, 4, kDbgSampleOut, P.logprob + row, -INFINITY);
    }
    return;
  }
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
  if (tid == 0) {
    const int32_t id = P.ids ? dload(P.dbg, 1, kDbgSampleLogits, P.ids + row * P.ld_ids + at) : at;
    dstore(P.dbg, 3, kDbgSampleOut, P.token + row, id);
    if (P.logprob) dstore(P.dbg, 4, kDbgSampleOut, P.logprob + row, static_cast<float>(log(kept(at) / total)));
  }
}

hipError_t launch_sample(const SamplePlan& p, const SampleArgs& a, hipStream_t st) {
  SampleParams P;
  P.logits = a.logits, P.ld = p.ld;
  P.ids = a.ids, P.ld_ids = p.ld_ids;
  P.u = a.u, P.set = a.params;
  P.token = a.token, P.logprob = a.logprob;
  P.V = static_cast<int32_t>(p.V);
  const uint64_t n = static_cast<uint64_t>(p.N);
  P.dbg = make_debug_check(reinterpret_cast<uint32_t*>(a.ws + kDebugWordOffset),
                           {{a.logits, ((n - 1) * p.ld + p.V) * type_bytes(p.type)},
                            {a.ids, a.ids ? ((n - 1) * p.ld_ids + p.V) * 4 : 0},
                            {a.u, n * 4},
                            {a.token, n * 4},
                            {a.logprob, a.logprob ? n * 4 : 0}});
  // V weights of at most 2^shift each stay below 2^63
  int shift = 46;
  while ((p.V >> (62 - shift)) > 0) --shift;
  TraceScope ts(st, "sample_row", 0.0, static_cast<double>(p.N) * p.V * type_bytes(p.type));
  auto* k = p.type == FKL_F32 ? k_sample_row<float> : p.type == FKL_BF16 ? k_sample_row<__bf16> : k_sample_row<_Float16>;
  constexpr int64_t kRowsPerLaunch = int64_t(1) << 21;  // grid x block stays below 2^32 threads
  for (int64_t r = 0; r < p.N; r += kRowsPerLaunch) {
    P.row0 = r;
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(std::min(p.N - r, kRowsPerLaunch))), dim3(kRowThreads), 0, st, P,
                       shift);
  }
  return hipGetLastError();
}

}  // namespace fkl
