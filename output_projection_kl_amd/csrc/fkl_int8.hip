// The 8-bit head on gfx950: rows quantised to int8 with one scale each
// (fkl_quantize), and out = a_scale b_scale (A B^T) + bias over int8 operands
// (fkl_project), A [M,K] and B [N,K] with k contiguous.
#include <algorithm>
#include <type_traits>

#include "fkl_decode.h"
#include "fkl_device.h"
#include "fkl_tiles.h"

namespace fkl {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// Quantisation
//
// q = rne(127 x / a) of the real quotient. t = p / a' with p = 127 x 2^-e and
// a' = a 2^-e (e the exponent of a, so neither over- nor underflows where it
// matters). p is exact: x has at most 11 significant bits (24 in fp32, where
// the whole computation is in 64 bits). t is formed by a reciprocal and one
// residual step, which leaves it within half a unit of the last place:
// halves, which fp32 (fp64) holds exactly, come out exactly, and any other
// quotient is at least 1 / (254 * 2047) = 1.9e-6 (2.3e-10 for 24 bits) of its
// value away from a half, more than 2^-24 (2^-53): the rounding to an integer
// is that of the real quotient.
//
// HBM bound: the row is read once, held in registers between the maximum and
// the rounding.
// ---------------------------------------------------------------------------

constexpr int kQuantThreads = 256;
constexpr int kQuantHeldBytes = 64;  // bytes of a row that a thread holds: 16 KiB rows stay in registers

template <class T>
struct QuantOf;

struct QuantScale32 {
  float c, a, inv;  // 127 * 2^-e, a * 2^-e, its reciprocal
  __device__ __forceinline__ explicit QuantScale32(float amax) {
    int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
    e = e < -119 ? -119 : e > 126 ? 126 : e;  // 127 * 2^-e and 2^-e stay normal numbers
    const float s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    c = 127.0f * s;
    a = amax * s;
    inv = 1.0f / a;
  }
  __device__ __forceinline__ int level(float x) const {
    const float p = x * c;
    const float t = p * inv;
    return static_cast<int>(rintf(fmaf(fmaf(-t, a, p), inv, t)));
  }
};

struct QuantScale64 {
  double a, inv;
  __device__ __forceinline__ explicit QuantScale64(float amax) : a(amax), inv(1.0 / static_cast<double>(amax)) {}
  __device__ __forceinline__ int level(float x) const {
    const double p = 127.0 * static_cast<double>(x);
    const double t = p * inv;
    return static_cast<int>(rint(fma(fma(-t, a, p), inv, t)));
  }
};

// A row's elements as bits whose unsigned order is that of the magnitudes (NaN
// above infinity above every number), four bytes at a time.
template <>
struct QuantOf<float> {
  using Scale = QuantScale64;
  static constexpr uint32_t kAbs = 0x7fffffffu;
  static constexpr uint32_t kInf = 0x7f800000u;
  __device__ static uint32_t wider(uint32_t m, uint32_t w) { return max(m, w & kAbs); }
  __device__ static uint32_t magnitude(uint32_t m) { return m; }
  __device__ static float value(uint32_t bits) { return __uint_as_float(bits); }
};

struct QuantHalves {
  using Scale = QuantScale32;
  static constexpr uint32_t kAbs = 0x7fff7fffu;
  __device__ static uint32_t wider(uint32_t m, uint32_t w) {
    return __builtin_bit_cast(
        uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m), __builtin_bit_cast(u16x2, w & kAbs)));
  }
  __device__ static uint32_t magnitude(uint32_t m) { return max(m & 0xffffu, m >> 16); }
};

template <>
struct QuantOf<__bf16> : QuantHalves {
  static constexpr uint32_t kInf = 0x7f80u;
  __device__ static float value(uint32_t bits) { return __uint_as_float(bits << 16); }
};

template <>
struct QuantOf<_Float16> : QuantHalves {
  static constexpr uint32_t kInf = 0x7c00u;
  __device__ static float value(uint32_t bits) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
  }
};

// The largest of m over the block, and the row's scale.
template <class T>
__device__ __forceinline__ uint32_t block_magnitude(uint32_t m, uint32_t* shared) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = QuantOf<T>::wider(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, 64)));
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 64; ++w) m = QuantOf<T>::wider(m, shared[w]);
  return QuantOf<T>::magnitude(m);
}

template <class T>
__device__ __forceinline__ float row_scale(uint32_t mag) {
  return mag >= QuantOf<T>::kInf ? __uint_as_float(0x7fc00000u) : QuantOf<T>::value(mag) / 127.0f;
}

// Levels of the 16 / sizeof(T) elements of one 16-byte piece, packed in bytes.
template <class T>
__device__ __forceinline__ void pack_levels(const typename QuantOf<T>::Scale& s, u32x4 v, uint32_t* out) {
  constexpr int kPerWord = 4 / sizeof(T);
#pragma unroll
  for (int o = 0; o < 4 / static_cast<int>(sizeof(T)); ++o) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = o * 4 + j;
      uint32_t bits = v[i / kPerWord];
      if constexpr (sizeof(T) == 2) bits = (i & 1) ? bits >> 16 : bits & 0xffffu;
      w |= (static_cast<uint32_t>(s.level(QuantOf<T>::value(bits))) & 0xffu) << (8 * j);
    }
    out[o] = w;
  }
}

// One workgroup per row, in pieces of 16 bytes of x; the row's last few
// elements one by one. Pieces are read and written at any alignment (the GPU
// splits an access that crosses a line). 128256 x 4096 bf16: 244 us, 6.45 TB/s
// read and written (281 us without the non-temporal hint of ONCE); 4096 x 2880
// bf16, which the caches hold: 10 us.
template <class T, bool ONCE>
__global__ __launch_bounds__(kQuantThreads) void k_quantize(const T* __restrict__ x, int64_t ldx, int cols,
                                                            int8_t* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scale) {
  __shared__ uint32_t shared[kQuantThreads / 64];
  constexpr int kPer = 16 / sizeof(T);
  constexpr int kHeld = kQuantHeldBytes / 16;
  constexpr int kWords = kPer / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
  typedef u32x4 AnyPiece __attribute__((aligned(1)));
  typedef Words AnyWords __attribute__((aligned(1)));
  const int64_t row = blockIdx.x;
  const T* const src = x + row * ldx;
  int8_t* const dst = q + row * ldq;
  const int n = cols / kPer;
  const int tail = n * kPer + threadIdx.x;  // this thread's element of the tail
  auto get = [&](int i) -> u32x4 {
    const AnyPiece* const at = reinterpret_cast<const AnyPiece*>(src + static_cast<int64_t>(i) * kPer);
    if constexpr (ONCE) return __builtin_nontemporal_load(at);
    else return *at;
  };
  auto element = [&](int i) -> uint32_t {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(uint32_t, src[i]);
    else return __builtin_bit_cast(uint16_t, src[i]);
  };
  u32x4 held[kHeld];
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int i = threadIdx.x + h * kQuantThreads;
    held[h] = i < n ? get(i) : u32x4{0, 0, 0, 0};
  }
  const uint32_t last = tail < cols ? element(tail) : 0u;
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = QuantOf<T>::wider(m, held[h][j]);
  m = QuantOf<T>::wider(m, last);
  for (int i = threadIdx.x + kHeld * kQuantThreads; i < n; i += kQuantThreads) {
    const u32x4 v = get(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) m = QuantOf<T>::wider(m, v[j]);
  }
  const uint32_t mag = block_magnitude<T>(m, shared);
  if (threadIdx.x == 0) scale[row] = row_scale<T>(mag);
  const bool zero = mag == 0 || mag >= QuantOf<T>::kInf;
  const typename QuantOf<T>::Scale s(zero ? 1.0f : QuantOf<T>::value(mag));
  auto put = [&](int i, u32x4 v) {
    uint32_t w[kWords];
    pack_levels<T>(s, v, w);
    Words out;
#pragma unroll
    for (int j = 0; j < kWords; ++j) out[j] = zero ? 0u : w[j];
    AnyWords* const at = reinterpret_cast<AnyWords*>(dst + static_cast<int64_t>(i) * kPer);
    if constexpr (ONCE) __builtin_nontemporal_store(out, at);
    else *at = out;
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int i = threadIdx.x + h * kQuantThreads;
    if (i < n) put(i, held[h]);
  }
  for (int i = threadIdx.x + kHeld * kQuantThreads; i < n; i += kQuantThreads) put(i, get(i));
  if (tail < cols) dst[tail] = zero ? int8_t(0) : static_cast<int8_t>(s.level(QuantOf<T>::value(last)));
}

template <class T>
static void launch_quantize_of(int64_t rows, int64_t cols, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                               float* scale, hipStream_t st) {
  constexpr int64_t kRowsPerLaunch = int64_t(1) << 23;  // grid x block stays below 2^32 threads
  // what the last-level cache cannot keep is better not brought there
  const int64_t bytes = rows * cols * static_cast<int64_t>(sizeof(T));
  auto* const k = bytes > kLastLevelBytes ? k_quantize<T, true> : k_quantize<T, false>;
  for (int64_t r = 0; r < rows; r += kRowsPerLaunch)
    hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(std::min(rows - r, kRowsPerLaunch))),
                       dim3(kQuantThreads), 0, st, static_cast<const T*>(x) + r * ldx, ldx, static_cast<int>(cols),
                       q + r * ldq, ldq, scale + r);
}

hipError_t launch_quantize(int64_t rows, int64_t cols, int type, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                           float* scale, hipStream_t st) {
  const double n = static_cast<double>(rows) * cols;
  TraceScope ts(st, "quantize", 0.0, n * (type_bytes(type) + 1) + 4.0 * rows);
  if (type == FKL_F32) launch_quantize_of<float>(rows, cols, x, ldx, q, ldq, scale, st);
  else if (type == FKL_BF16) launch_quantize_of<__bf16>(rows, cols, x, ldx, q, ldq, scale, st);
  else launch_quantize_of<_Float16>(rows, cols, x, ldx, q, ldq, scale, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Product
// ---------------------------------------------------------------------------

// Rows of K bytes at any stride and alignment copied to rows of row16 bytes
// (16-byte aligned, a multiple of 16); the bytes past K are zeroed. HBM bound:
// 32003 x 2887 of stride 2889, 29 us, 6.4 TB/s read and written (92 us a byte at
// a time).
__global__ __launch_bounds__(256) void k_copy_rows(const int8_t* __restrict__ src, int64_t ld, int64_t rows, int K,
                                                   int row16, int8_t* __restrict__ dst, DebugCheck dbg) {
  const int pieces = row16 / 16;
  const int64_t n = rows * pieces;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    const int64_t r = i / pieces;
    const int k0 = static_cast<int>(i - r * pieces) * 16;
    const int8_t* s = src + r * ld + k0;
    u32x4 v{0, 0, 0, 0};
    if (k0 + 16 <= K) {
      typedef u32x4 AnyPiece __attribute__((aligned(1)));
      if (dcheck_range(dbg, 0, kDbgProjectOperand, s, 16)) v = *reinterpret_cast<const AnyPiece*>(s);
    } else {
      for (int j = 0; k0 + j < K; ++j)
        v[j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(dload(dbg, 0, kDbgProjectOperand, s + j))) << (8 * (j % 4));
    }
    dstore(dbg, 1, kDbgProjectWork, reinterpret_cast<u32x4*>(dst + i * 16), v);
  }
}

struct ProjectParams {
  Operand A, B;  // rows of int8 seen as 16-bit pairs: ld and k_lim count pairs
  int32_t K;
  const float *a_scale, *b_scale, *bias;
  void* out;
  int64_t ldo, M, N;
  int32_t mblocks, nblocks;
  // Split contraction: split s covers the stages of k_split bytes from s k_split
  // on, and leaves its sums (T = int32_t) at out + s split_out.
  int32_t splits, k_split;
  int64_t split_out;
  DebugCheck dbg;  // debug build: span 0 = out, 1 = A, 2 = B, 3 = a_scale, 4 = b_scale, 5 = bias
};

// One output element: the sum times a_scale (one rounding after the sum's
// conversion), then one fused multiply-add, rounded to the output type.
template <class T>
__device__ __forceinline__ T scaled(int32_t sum, float sa, float sb, float bias) {
  float v = fmaf(static_cast<float>(sum) * sa, sb, bias);
  // the fp32 result stands by itself: the compiler may otherwise round to fp16
  // within the multiply-add in some of the kernels, and they would differ
  asm("" : "+v"(v));
  return static_cast<T>(v);
}

template <>
__device__ __forceinline__ int32_t scaled<int32_t>(int32_t sum, float, float, float) {
  return sum;
}

// Bytes `valid` .. of a lane's 16 cleared.
__device__ __forceinline__ i32x4 keep_bytes(i32x4 v, int valid) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = valid - 4 * j;
    v[j] &= n >= 4 ? -1 : n <= 0 ? 0 : (1 << (8 * n)) - 1;
  }
  return v;
}

// ---- few output elements ---------------------------------------------------
//
// 16 rows of A against 16 columns of the output (rows of B) at a time, the
// contraction split over the workgroup's 8 waves: wave w takes the F 64-byte
// fragments from w F on of each span of 512 F bytes. A and B go from memory
// straight to the MFMA operands (lane l: row l & 15, 16 bytes at 16 (l >> 4)),
// the next tile's B while this one's is used; A's fragments stay in registers
// where one span covers K. The waves' partial sums meet in LDS. Latency bound:
// all of a tile's reads are on their way at once, where a block tile goes
// through its contraction stage by stage (5 x 1024 x 1024: 3 against 5 us).
constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyThreads = 64 * kSkinnyWaves;

template <class T, int F>
__global__ __launch_bounds__(kSkinnyThreads) void k_project_skinny(ProjectParams P, int spans) {
  __shared__ i32x4 part[2][kSkinnyWaves][64];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 16;
  const int8_t* const a = reinterpret_cast<const int8_t*>(P.A.base);
  const int8_t* const b = reinterpret_cast<const int8_t*>(P.B.base);
  const int64_t lda = P.A.ld * 2, ldb = P.B.ld * 2;
  const int K16 = static_cast<int>(P.A.k_lim) * 2;
  const int k_lane = wave * (F * 64) + (lane >> 4) * 16;

  // A's bytes past K and rows past M are zero; what is read for B there then
  // does not matter, and comes from inside B.
  i32x4 fa[F];
  const int64_t m_lane = m0 + (lane & 15);
  const int8_t* const a_row = a + (m_lane < P.M ? m_lane : 0) * lda;
  auto load_a = [&](int span) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int k = span * (kSkinnyWaves * F * 64) + k_lane + f * 64;
      const i32x4 v = dload(P.dbg, 1, kDbgProjectOperand, reinterpret_cast<const i32x4*>(a_row + (k < K16 ? k : 0)));
      fa[f] = keep_bytes(v, m_lane < P.M ? P.K - k : 0);
    }
  };
  auto load_b = [&](int tile, int span, i32x4 (&fb)[F]) {
    int64_t n = static_cast<int64_t>(tile) * 16 + (lane & 15);
    n = n < P.N ? n : P.N - 1;
    const int8_t* const row = b + n * ldb;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int k = span * (kSkinnyWaves * F * 64) + k_lane + f * 64;
      fb[f] = dload(P.dbg, 2, kDbgProjectOperand, reinterpret_cast<const i32x4*>(row + (k < K16 ? k : 0)));
    }
  };
  i32x4 acc;
  auto mma = [&](const i32x4 (&fb)[F]) {
#pragma unroll
    for (int f = 0; f < F; ++f) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[f], fb[f], acc, 0, 0, 0);
  };
  // The tile's sums from the waves' accumulators (lane l: column l & 15, rows 4 (l >> 4) .. + 3).
  auto finish = [&](int tile, int turn) {
    part[turn][wave][lane] = acc;
    __syncthreads();
    const int row = tid >> 4, col = tid & 15;
    const int64_t m = m0 + row, n = static_cast<int64_t>(tile) * 16 + col;
    if (tid < 256 && m < P.M && n < P.N) {
      int32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kSkinnyWaves; ++w)
        sum += reinterpret_cast<const int32_t*>(&part[turn][w][(row >> 2) * 16 + col])[row & 3];
      const float sa = dload(P.dbg, 3, kDbgProjectOperand, P.a_scale + m);
      const float sb = dload(P.dbg, 4, kDbgProjectOperand, P.b_scale + n);
      const float bias = P.bias ? dload(P.dbg, 5, kDbgProjectOperand, P.bias + n) : 0.0f;
      dstore(P.dbg, 0, kDbgProjectOut, static_cast<T*>(P.out) + m * P.ldo + n, scaled<T>(sum, sa, sb, bias));
    }
  };

  const int step = gridDim.x;
  int turn = 0;  // the two halves of `part` take turns: one barrier per tile
  if (spans == 1) {
    load_a(0);
    i32x4 fb[2][F];
    int tile = blockIdx.x;
    load_b(tile, 0, fb[0]);
    while (true) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (tile + step < P.nblocks) load_b(tile + step, 0, fb[1 - h]);
        acc = i32x4{0, 0, 0, 0};
        mma(fb[h]);
        finish(tile, h);
        tile += step;
        if (tile >= P.nblocks) return;
      }
    }
  }
  for (int tile = blockIdx.x; tile < P.nblocks; tile += step, turn ^= 1) {
    acc = i32x4{0, 0, 0, 0};
    for (int span = 0; span < spans; ++span) {
      i32x4 fb[F];
      load_b(tile, span, fb);
      load_a(span);
      mma(fb);
    }
    finish(tile, turn);
  }
}

// ---- block tiles ----------------------------------------------------------
//
// TM x TN of the output on WM x WN waves, through a ring of S LDS stages of
// 128 bytes of the contraction per row: two v_mfma_i32_16x16x64_i8 steps. The
// stages are filled by direct global->LDS loads of 16 bytes per lane, eight
// lanes on one row's 128 bytes: whole cache lines. (With 64-byte stage rows,
// as the bf16 tiles have them, each line is asked for twice, and the loads
// alone took 210 of the 287 us of a 8192 x 8192 x 4096 product.)
//
// LDS: row r of a stage at 128 r, its 16-byte chunk c at physical chunk c ^
// ((r >> 1) & 7): a fragment's 16 rows then lie on 16 distinct 16-byte groups
// of the 256 bytes that the banks span. Fragments of A and B use the same
// assignment of bytes to lanes, so any order of k within a step gives the same
// sum; in the last stage A's bytes past K are cleared, and what B holds there
// does not matter.
constexpr int kIntStageK = 128;

template <int TM_, int TN_, int WM_, int WN_, int S_, ProjectRead READ_ = kReadPlain>
struct IntTile {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, S = S_;
  template <ProjectRead READ>
  using As = IntTile<TM, TN, WM, WN, S, READ>;
  // B's rows by whole lines: stage t of a row starts at the line boundary at or
  // below its 128 t-th byte, and step t lies in stages t and t + 1
  static constexpr bool kByLines = READ_ == kReadOnceByLines;
  static constexpr int kPolicy = READ_ == kReadPlain ? 0 : 2;  // of B's load instructions: 2 = non-temporal
  static constexpr int kAhead = kByLines ? 2 : 1;               // stages in LDS from a step's first one on
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int XA = TM / WM / 16;  // 16-row fragments of a wave
  static constexpr int XB = TN / WN / 16;
  static constexpr int kStageA = TM * kIntStageK;
  static constexpr int kStage = (TM + TN) * kIntStageK;
  static constexpr int LA = (TM / 8 + kWaves - 1) / kWaves;  // loads per lane per stage, 8 rows a wave each
  static constexpr int LB = (TN / 8 + kWaves - 1) / kWaves;
  static constexpr int kDma = LA + LB;
  // where waves that have no rows left load to, so that every wave's count of loads is the same
  static constexpr bool kSpare = LA * kWaves * 8 != TM || LB * kWaves * 8 != TN;
  static constexpr int kRing = S * kStage + (kSpare ? 1024 * kWaves : 0);
  static_assert(TM % (16 * WM) == 0 && TN % (16 * WN) == 0, "whole fragments");
  static_assert(S > kAhead, "a stage to load while those are used");
  // the epilogue's staging: rows of out_cols columns of the output type, 16 bytes apart from each other
  static constexpr int out_cols(int size) { return TN * size < 512 ? TN : 512 / size; }
  static constexpr int out_pitch(int size) { return out_cols(size) * size + 16; }
  static constexpr int lds(int size) {
    return kRing > TM * out_pitch(size) ? kRing : TM * out_pitch(size);
  }
};

// One operand's stage loads of a wave: load j covers rows 8 (wave L + j) .. + 7
// of the tile's R rows.
template <int L>
struct IntSrc {
  const int8_t* base;
  int32_t bytes;  // of the rows inside the operand; what lies past them reads as zero
  uint32_t off[L];
  int32_t lead[L];  // bytes of the row's stage 0 in front of the row
  int32_t chunk;    // first byte of the lane's chunk within the stage
  int32_t k_lim;
};

// Bytes from the line boundary at or below row r's start up to it: the same
// for r and r + 16, since the rows' stride is a multiple of 16 bytes.
__device__ __forceinline__ int line_lead(const Operand& op, int64_t row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(op.base) + static_cast<uint64_t>(row * op.ld * 2)) &
                          (kIntStageK - 1));
}

template <int R, int L, bool LINES>
__device__ __forceinline__ IntSrc<L> int_src(const Operand& op, int64_t row0, int wave, int lane) {
  IntSrc<L> s;
  const OperandView v = plain_view(op, row0, R);
  s.base = reinterpret_cast<const int8_t*>(v.base);
  s.bytes = static_cast<int32_t>(v.bytes);
#pragma unroll
  for (int j = 0; j < L; ++j) {
    const int r = (wave * L + j) * 8 + (lane >> 3);
    s.off[j] = r < R ? static_cast<uint32_t>(r * op.ld * 2) : kOob;
    s.lead[j] = LINES ? line_lead(op, row0 + r) : 0;
  }
  s.chunk = (lane & 7) << 4;
  s.k_lim = static_cast<int32_t>(op.k_lim) * 2;
  return s;
}

// Issues stage kt of one operand into its LDS region; every lane reads out of
// range (zeros, no memory access) where live is false.
template <int R, int L, int POLICY>
__device__ __forceinline__ void issue_int(const IntSrc<L>& s, int kt, bool live, char* region, char* spare, int wave,
                                          int lane) {
  const __amdgpu_buffer_rsrc_t rsrc =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(s.base), 0, s.bytes, 0x00020000);
#pragma unroll
  for (int j = 0; j < L; ++j) {
    const int block = wave * L + j;
    const int r = block * 8 + (lane >> 3);
    const int k = kt * kIntStageK + (s.chunk ^ (((r >> 1) & 7) << 4)) - s.lead[j];
    uint32_t off = s.off[j] + static_cast<uint32_t>(k);
    if (!live || k < 0 || k >= s.k_lim || s.off[j] == kOob) off = kOob;
    char* dst = block * 8 < R ? region + block * 1024 : spare + wave * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (FKL_LDS void*)dst, 16, static_cast<int>(off), 0, 0, POLICY);
  }
}

// Fragment of 16 rows x 64 bytes, step kk of a stage: lane l receives row l &
// 15, bytes 16 (l >> 4) .. + 15.
__device__ __forceinline__ i32x4 int_frag(const char* region, int row0, int kk, int lane) {
  const int r = row0 + (lane & 15);
  const int c = kk * 4 + (lane >> 4);
  return *reinterpret_cast<const i32x4*>(region + r * kIntStageK + ((c ^ ((r >> 1) & 7)) << 4));
}

// acc = A[m0 : m0 + TM] B[n0 : n0 + TN]^T, with B as the MFMA's first operand:
// lane l then holds four consecutive columns 4 (l >> 4) .. + 3 of row l & 15 of
// each 16 x 16 block. Two sets of fragments: while the
// MFMAs of one step run, the fragments of the next are read, so that the
// matrix pipe and LDS work at once; the order of issue is fixed by hand (left
// alone, the compiler gathers the reads at the end). Per stage one barrier, at
// its second step: every wave holds all of its fragments of the stage, whose
// place then takes the loads of stage kt + S, and has waited for its own loads
// of stage kt + 1. (LDS reads come before the loads: the compiler makes a read
// that follows a global->LDS load wait for it.)
template <class C>
__device__ __forceinline__ void int8_mainloop(const Operand& A, const Operand& B, int64_t m0, int64_t n0, int K,
                                              i32x4 (&acc)[C::XA][C::XB], char* lds) {
  constexpr int S = C::S;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int am = (wave / C::WN) * (C::XA * 16);
  const int bn = (wave % C::WN) * (C::XB * 16);
  const int n_stages = (K + kIntStageK - 1) / kIntStageK;
  const IntSrc<C::LA> sa = int_src<C::TM, C::LA, false>(A, m0, wave, lane);
  const IntSrc<C::LB> sb = int_src<C::TN, C::LB, C::kByLines>(B, n0, wave, lane);
  // of step kk: this lane's place in the stage that holds it, and which that is
  int b_at[2];
  bool b_next[2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const int r = lane & 15;
    const int at = kk * 64 + (lane >> 4) * 16 + line_lead(B, n0 + r);
    b_at[kk] = C::kStageA + (bn + r) * kIntStageK + (((at >> 4) & 7) ^ ((r >> 1) & 7)) * 16;
    b_next[kk] = at >= kIntStageK;
  }
  char* const spare = lds + S * C::kStage;
  auto issue = [&](int kt) {
    char* place = lds + (kt % S) * C::kStage;
    issue_int<C::TM, C::LA, 0>(sa, kt, kt < n_stages, place, spare, wave, lane);
    issue_int<C::TN, C::LB, C::kPolicy>(sb, kt, kt < n_stages + C::kByLines, place + C::kStageA, spare, wave, lane);
  };
  struct Set {
    i32x4 a[C::XA], b[C::XB];
  } f[2];
  auto read = [&](Set& t, int kt, int kk) {
    const char* st = lds + (kt % S) * C::kStage;
#pragma unroll
    for (int x = 0; x < C::XA; ++x) t.a[x] = int_frag(st, am + x * 16, kk, lane);
#pragma unroll
    for (int y = 0; y < C::XB; ++y) {
      if constexpr (C::kByLines) {
        const char* const at = b_next[kk] ? lds + ((kt + 1) % S) * C::kStage : st;
        t.b[y] = *reinterpret_cast<const i32x4*>(at + b_at[kk] + y * 16 * kIntStageK);
      } else {
        t.b[y] = int_frag(st + C::kStageA, bn + y * 16, kk, lane);
      }
    }
  };
  auto mma = [&](const Set& t) {
#pragma unroll
    for (int x = 0; x < C::XA; ++x)
#pragma unroll
      for (int y = 0; y < C::XB; ++y)
        acc[x][y] = __builtin_amdgcn_mfma_i32_16x16x64_i8(t.b[y], t.a[x], acc[x][y], 0, 0, 0);
  };
#pragma unroll
  for (int x = 0; x < C::XA; ++x)
#pragma unroll
    for (int y = 0; y < C::XB; ++y) acc[x][y] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int p = 0; p < S; ++p) issue(p);
  wait_vmcnt<(S - C::kAhead) * C::kDma>();
  block_barrier();
  read(f[0], 0, 0);
  constexpr int kMfma = C::XA * C::XB;
  constexpr int kReads = C::XA + C::XB;
  constexpr int kFirst = kMfma >= kReads ? kMfma / kReads : 1;  // MFMAs per fragment read
  constexpr int kSecond = kMfma >= kReads + C::kDma ? kMfma / (kReads + C::kDma) : 1;  // and with the loads
  for (int kt = 0; kt + 1 < n_stages; ++kt) {
    __builtin_amdgcn_sched_barrier(0);
    read(f[1], kt, 1);
    mma(f[0]);
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kFirst, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<(S - 1 - C::kAhead) * C::kDma>();
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    block_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(f[0], kt + 1, 0);
    issue(kt + S);
    mma(f[1]);
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kSecond, 0);
    }
#pragma unroll
    for (int i = 0; i < C::kDma; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kSecond, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  const int last = K - (n_stages - 1) * kIntStageK - 16 * (lane >> 4);  // bytes from the lane's chunk on
  read(f[1], n_stages - 1, 1);
#pragma unroll
  for (int x = 0; x < C::XA; ++x) f[0].a[x] = keep_bytes(f[0].a[x], last), f[1].a[x] = keep_bytes(f[1].a[x], last - 64);
  mma(f[0]);
  mma(f[1]);
  wait_vmcnt<0>();
  block_barrier();
}

// One output tile per workgroup. MFMA bound for the large tiles: 8192 x 128256 x
// 4096 into bf16 takes 3.6 ms, 2390 TOP/s (5030 at the full rate; the GPU's clock
// falls with the load). HBM bound for few rows: 1 x 201088 x 2880, 96 us, 6.0
// TB/s; 48 x 128256 x 4096, 103 us, 5.2 TB/s, where the tiles' starts and ends
// show. The results are staged in LDS in the output's type and stored as whole lines: stored
// from the registers (32 bytes of a row at a time) they took a 8192 x 128256 x
// 4096 product from 4.09 to 4.58 ms.
template <class T, class C>
__global__ __launch_bounds__(C::kThreads) void k_project(ProjectParams P) {
  __shared__ __align__(16) char lds[C::lds(sizeof(T))];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  int mbi, nbi;
  const int tiles = P.mblocks * P.nblocks;
  const int at = xcd_contiguous(blockIdx.x, tiles * P.splits);
  const int split = at / tiles;
  grouped_tile(at - split * tiles, P.mblocks, P.nblocks, 8, mbi, nbi);
  const int64_t m0 = static_cast<int64_t>(mbi) * C::TM;
  const int64_t n0 = static_cast<int64_t>(nbi) * C::TN;
  const int k0 = split * P.k_split;
  const Operand A = k_window<false>(P.A, k0 / 2, P.k_split / 2);
  const Operand B = k_window<false>(P.B, k0 / 2, P.k_split / 2);
  i32x4 acc[C::XA][C::XB];
  dcheck_operand(P.dbg, 1, A, m0, C::TM, false);
  dcheck_operand(P.dbg, 2, B, n0, C::TN, false);
  int8_mainloop<C>(A, B, m0, n0, min(P.K - k0, P.k_split), acc, lds);
  constexpr int kCols = C::out_cols(sizeof(T));
  constexpr int kPitch = C::out_pitch(sizeof(T));
  typedef T T4 __attribute__((ext_vector_type(4)));
  const int m_wave = (wave / C::WN) * (C::XA * 16) + (lane & 15);  // of this lane's rows within the tile
  const int n_wave = (wave % C::WN) * (C::XB * 16) + 4 * (lane >> 4);
  float sa[C::XA];
#pragma unroll
  for (int x = 0; x < C::XA; ++x) {
    const int64_t m = m0 + m_wave + x * 16;
    sa[x] = std::is_same<T, int32_t>::value || m >= P.M ? 0.0f : dload(P.dbg, 3, kDbgProjectOperand, P.a_scale + m);
  }
  T* const out = static_cast<T*>(P.out) + split * P.split_out + m0 * P.ldo + n0;
  const int rmax = static_cast<int>(min<int64_t>(C::TM, P.M - m0));
#pragma unroll
  for (int c0 = 0; c0 < C::TN; c0 += kCols) {
    const int cmax = static_cast<int>(min<int64_t>(kCols, P.N - n0 - c0));
    if (cmax <= 0) break;
#pragma unroll
    for (int y = 0; y < C::XB; ++y) {
      const int col = n_wave + y * 16 - c0;
      if (col < 0 || col >= kCols) continue;  // the same for the whole wave
      float sb[4], bias[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = !std::is_same<T, int32_t>::value && col + j < cmax;
        sb[j] = in ? dload(P.dbg, 4, kDbgProjectOperand, P.b_scale + n0 + c0 + col + j) : 0.0f;
        bias[j] = in && P.bias ? dload(P.dbg, 5, kDbgProjectOperand, P.bias + n0 + c0 + col + j) : 0.0f;
      }
#pragma unroll
      for (int x = 0; x < C::XA; ++x)
        *reinterpret_cast<T4*>(lds + (m_wave + x * 16) * kPitch + col * static_cast<int>(sizeof(T))) =
            T4{scaled<T>(acc[x][y][0], sa[x], sb[0], bias[0]), scaled<T>(acc[x][y][1], sa[x], sb[1], bias[1]),
               scaled<T>(acc[x][y][2], sa[x], sb[2], bias[2]), scaled<T>(acc[x][y][3], sa[x], sb[3], bias[3])};
    }
    __syncthreads();
    // 16 bytes of a row per lane, at 16-byte boundaries of the output: the
    // staged row is read `mis` bytes before the piece's own start where rows do
    // not start at such a boundary, in words, shifted by half a word if need be.
    constexpr int kSize = static_cast<int>(sizeof(T));
    constexpr int kPieces = kCols * kSize / 16;
    auto store_rows = [&](auto at_boundary) {
      constexpr int kAcross = kPieces + (at_boundary ? 0 : 1);
      constexpr int kDown = C::kThreads / kAcross;
      const int b = (tid % kAcross) * 16;
      for (int r = tid / kAcross; r < rmax && tid < kAcross * kDown; r += kDown) {
        char* const row = reinterpret_cast<char*>(out + r * P.ldo + c0);
        const int mis = at_boundary ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
        const int b0 = b - mis;  // the piece's first byte in the row
        const char* const from = lds + r * kPitch;
        if (b0 >= 0 && b0 + 16 <= cmax * kSize) {
          u32x4 v;
          if (mis == 0) {
            v = *reinterpret_cast<const u32x4*>(from + b0);
          } else {
            const uint32_t* const w = reinterpret_cast<const uint32_t*>(from + (b0 & ~3));
            v = u32x4{w[0], w[1], w[2], w[3]};
            if (kSize == 2 && (b0 & 2)) {
              const uint32_t next = w[4];
              v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16 | next << 16};
            }
          }
          dstore(P.dbg, 0, kDbgProjectOut, reinterpret_cast<u32x4*>(row + b0), v);
        } else {
          for (int e = max(b0, 0); e < min(b0 + 16, cmax * kSize); e += kSize)
            dstore(P.dbg, 0, kDbgProjectOut, reinterpret_cast<T*>(row + e), *reinterpret_cast<const T*>(from + e));
        }
      }
    };
    if (P.ldo * kSize % 16 == 0 && reinterpret_cast<uintptr_t>(P.out) % 16 == 0)
      store_rows(std::integral_constant<bool, true>());
    else
      store_rows(std::integral_constant<bool, false>());
    if (c0 + kCols < C::TN) __syncthreads();
  }
}

// The sums of a split contraction added up, scaled and rounded. Launch bound:
// the sums come from the cache (100 x 65 x 20011 in 14 us with the split product).
template <class T>
__global__ __launch_bounds__(256) void k_project_join(ProjectParams P, const int32_t* __restrict__ sums, int64_t ld) {
  const int64_t quads = (P.N + 3) / 4;
  const int64_t total = P.M * quads;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t m = i / quads;
    const int64_t n = (i - m * quads) * 4;
    i32x4 sum{0, 0, 0, 0};
    for (int s = 0; s < P.splits; ++s) sum += *reinterpret_cast<const i32x4*>(sums + s * P.split_out + m * ld + n);
    const float sa = dload(P.dbg, 3, kDbgProjectOperand, P.a_scale + m);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n + j >= P.N) break;
      const float sb = dload(P.dbg, 4, kDbgProjectOperand, P.b_scale + n + j);
      const float bias = P.bias ? dload(P.dbg, 5, kDbgProjectOperand, P.bias + n + j) : 0.0f;
      dstore(P.dbg, 0, kDbgProjectOut, static_cast<T*>(P.out) + m * P.ldo + n + j, scaled<T>(sum[j], sa, sb, bias));
    }
  }
}

using Tile256 = IntTile<256, 256, 2, 4, 2>;
using Tile256x128 = IntTile<256, 128, 4, 2, 3>;
using Tile128x256 = IntTile<128, 256, 2, 4, 3>;
using Tile128 = IntTile<128, 128, 2, 2, 2>;
using Tile64x128 = IntTile<64, 128, 2, 2, 3>;
using Tile64 = IntTile<64, 64, 2, 2, 3>;
using Tile32x64 = IntTile<32, 64, 1, 4, 4>;
using Tile16x64 = IntTile<16, 64, 1, 4, 4>;

template <class T, class C>
static void launch_tiles(ProjectParams P, hipStream_t st) {
  P.mblocks = static_cast<int32_t>(ceil_div(P.M, C::TM));
  P.nblocks = static_cast<int32_t>(ceil_div(P.N, C::TN));
  hipLaunchKernelGGL((k_project<T, C>), dim3(static_cast<unsigned>(P.mblocks) * P.nblocks * P.splits),
                     dim3(C::kThreads), 0, st, P);
}

template <class T>
static void launch_skinny(ProjectParams P, hipStream_t st) {
  P.nblocks = static_cast<int32_t>(ceil_div(P.N, 16));
  P.mblocks = static_cast<int32_t>(ceil_div(P.M, 16));
  const int per_wave = static_cast<int>(ceil_div(P.K, 64 * kSkinnyWaves));
  // as many workgroups as fit on the CUs at once, in all
  const int resident = 2 * kTargetBlocks;
  const dim3 grid(static_cast<unsigned>(std::min(P.nblocks, std::max(1, resident / P.mblocks))),
                  static_cast<unsigned>(P.mblocks));
  const dim3 block(kSkinnyThreads);
  if (per_wave <= 2) hipLaunchKernelGGL((k_project_skinny<T, 2>), grid, block, 0, st, P, 1);
  else if (per_wave <= 4) hipLaunchKernelGGL((k_project_skinny<T, 4>), grid, block, 0, st, P, 1);
  else
    hipLaunchKernelGGL((k_project_skinny<T, 8>), grid, block, 0, st, P, static_cast<int>(ceil_div(per_wave, 8)));
}

template <class T, class C>
static void launch_read(ProjectRead read, const ProjectParams& P, hipStream_t st) {
  if constexpr (C::TM <= kProjectLinesRows)
    if (read == kReadOnceByLines) return launch_tiles<T, typename C::template As<kReadOnceByLines>>(P, st);
  if (read == kReadOnce) return launch_tiles<T, typename C::template As<kReadOnce>>(P, st);
  launch_tiles<T, C>(P, st);
}

template <class T>
static void launch_shape(const ProjectPlan& p, ProjectRead read, const ProjectParams& P, hipStream_t st) {
  switch (p.shape) {
    case kProjectSkinny: return launch_skinny<T>(P, st);
    case kProject16x64: return launch_read<T, Tile16x64>(read, P, st);
    case kProject32x64: return launch_read<T, Tile32x64>(read, P, st);
    case kProject64: return launch_tiles<T, Tile64>(P, st);
    case kProject64x128: return launch_read<T, Tile64x128>(read, P, st);
    case kProject128: return launch_tiles<T, Tile128>(P, st);
    case kProject128x256: return launch_read<T, Tile128x256>(read, P, st);
    case kProject256x128: return launch_tiles<T, Tile256x128>(P, st);
    case kProject256: return launch_read<T, Tile256>(read, P, st);
  }
}

template <class T>
static void launch_product(const ProjectPlan& p, ProjectRead read, ProjectParams P, char* ws, hipStream_t st) {
  if (p.splits == 1) return launch_shape<T>(p, read, P, st);
  // sums of each split, then their join; only the 64 x 64 tiles are split
  ProjectParams Q = P;
  int32_t* const sums = reinterpret_cast<int32_t*>(ws + p.off_sums);
  const int64_t ld = round_up(p.N, 4);
  Q.out = sums;
  Q.ldo = ld;
  P.splits = Q.splits = p.splits;
  P.split_out = Q.split_out = p.M * ld;
  Q.k_split = static_cast<int32_t>(p.k_split);
  Q.dbg = P.dbg;
#ifdef FKL_DEBUG
  Q.dbg.s[0] = DebugSpan{reinterpret_cast<const char*>(sums), static_cast<uint64_t>(p.splits) * p.M * ld * 4};
#endif
  launch_tiles<int32_t, Tile64>(Q, st);
  const int64_t grid = std::min<int64_t>(ceil_div(p.M * (ld / 4), 256), 4096);
  hipLaunchKernelGGL(k_project_join<T>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, P, sums, ld);
}

hipError_t launch_project(const ProjectPlan& p, const ProjectArgs& g, hipStream_t st) {
  const int row16 = static_cast<int>(round_up(p.K, 16));
  uint32_t* word = reinterpret_cast<uint32_t*>(g.ws + kDebugWordOffset);
  const int8_t* a = static_cast<const int8_t*>(g.a);
  const int8_t* b = g.b;
  int64_t lda = p.lda, ldb = p.ldb;
  const float* a_scale = g.a_scale;
  auto copy = [&](const int8_t* src, int64_t ld, int64_t rows, int8_t* dst) {
    const uint64_t pieces = static_cast<uint64_t>(rows) * row16 / 16;
    const unsigned grid = static_cast<unsigned>(std::min<uint64_t>((pieces + 255) / 256, 8192));
    TraceScope ts(st, "project_copy", 0.0, static_cast<double>(rows) * (p.K + row16));
    hipLaunchKernelGGL(k_copy_rows, dim3(grid), dim3(256), 0, st, src, ld, rows, static_cast<int>(p.K), row16, dst,
                       make_debug_check(word, {{src, static_cast<uint64_t>((rows - 1) * ld + p.K)}, {dst, static_cast<uint64_t>(rows) * row16}}));
  };
  if (p.a_type != FKL_I8) {
    int8_t* q = reinterpret_cast<int8_t*>(g.ws + p.off_a);
    float* s = reinterpret_cast<float*>(g.ws + p.off_a_scale);
    const hipError_t e = launch_quantize(p.M, p.K, p.a_type, g.a, p.lda, q, p.row_a, s, st);
    if (e != hipSuccess) return e;
    a = q, lda = p.row_a, a_scale = s;
  } else if (p.a_copied) {
    int8_t* c = reinterpret_cast<int8_t*>(g.ws + p.off_a);
    copy(a, lda, p.M, c);
    a = c, lda = row16;
  }
  if (p.b_copied) {
    int8_t* c = reinterpret_cast<int8_t*>(g.ws + p.off_b);
    copy(b, ldb, p.N, c);
    b = c, ldb = row16;
  }
  ProjectParams P;
  P.A = Operand{reinterpret_cast<const uint16_t*>(a), lda / 2, p.M, row16 / 2};
  P.B = Operand{reinterpret_cast<const uint16_t*>(b), ldb / 2, p.N, row16 / 2};
  P.K = static_cast<int32_t>(p.K);
  P.splits = 1;
  P.k_split = static_cast<int32_t>(round_up(p.K, kIntStageK));
  P.split_out = 0;
  P.a_scale = a_scale, P.b_scale = g.b_scale, P.bias = g.bias;
  P.out = g.out;
  P.ldo = p.ldo, P.M = p.M, P.N = p.N;
  P.mblocks = P.nblocks = 0;  // by the variant
  const uint64_t out_bytes = static_cast<uint64_t>((p.M - 1) * p.ldo + p.N) * type_bytes(p.out_type);
  P.dbg = make_debug_check(word, {{g.out, out_bytes},
                                  {a, static_cast<uint64_t>((p.M - 1) * lda + row16)},
                                  {b, static_cast<uint64_t>((p.N - 1) * ldb + row16)},
                                  {a_scale, static_cast<uint64_t>(p.M) * 4},
                                  {g.b_scale, static_cast<uint64_t>(p.N) * 4},
                                  {g.bias, static_cast<uint64_t>(p.N) * 4}});
  const double flops = 2.0 * p.M * static_cast<double>(p.N) * p.K;
  const double bytes = static_cast<double>(p.M) * p.K + static_cast<double>(p.N) * p.K +
                       static_cast<double>(p.M) * p.N * type_bytes(p.out_type);
  const bool at_lines = ldb % 128 == 0 && reinterpret_cast<uintptr_t>(b) % 128 == 0;
  const ProjectRead read = !p.once ? kReadPlain
                           : at_lines ? kReadOnce
                           : p.shape <= kProject32x64 ? kReadOnceByLines
                                                      : kReadPlain;
  static const char* const kNames[] = {"project_16x16",   "project_16x64",   "project_32x64",   "project_64x64",
                                       "project_64x128",  "project_128x128", "project_128x256", "project_256x128",
                                       "project_256x256"};
  TraceScope ts(st, p.splits > 1 ? "project_split" : kNames[p.shape], flops, bytes);
  if (p.out_type == FKL_F32) launch_product<float>(p, read, P, g.ws, st);
  else if (p.out_type == FKL_BF16) launch_product<__bf16>(p, read, P, g.ws, st);
  else launch_product<_Float16>(p, read, P, g.ws, st);
  return hipGetLastError();
}

}  // namespace fkl
