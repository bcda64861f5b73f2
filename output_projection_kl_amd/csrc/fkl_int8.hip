// The 8-bit head on gfx950: rows quantised to int8 with one scale each
// (fkl_quantize), and out = a_scale b_scale (A B^T) + bias over int8 operands
// (fkl_project), A [M,K] and B [N,K] with k contiguous.
#include <algorithm>

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

// One workgroup per row, rows of whole 16-byte pieces (x 16-byte aligned, cols
// a multiple of 16 / sizeof(T), q aligned to the piece's levels).
template <class T>
__global__ __launch_bounds__(kQuantThreads) void k_quantize(const T* __restrict__ x, int64_t ldx, int cols,
                                                            int8_t* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ scale) {
  __shared__ uint32_t shared[kQuantThreads / 64];
  constexpr int kPer = 16 / sizeof(T);
  constexpr int kHeld = kQuantHeldBytes / 16;
  const int64_t row = blockIdx.x;
  const u32x4* src = reinterpret_cast<const u32x4*>(x + row * ldx);
  int8_t* dst = q + row * ldq;
  const int n = cols / kPer;
  u32x4 held[kHeld];
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int i = threadIdx.x + h * kQuantThreads;
    held[h] = i < n ? src[i] : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = QuantOf<T>::wider(m, held[h][j]);
  for (int i = threadIdx.x + kHeld * kQuantThreads; i < n; i += kQuantThreads) {
    const u32x4 v = src[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) m = QuantOf<T>::wider(m, v[j]);
  }
  const uint32_t mag = block_magnitude<T>(m, shared);
  if (threadIdx.x == 0) scale[row] = row_scale<T>(mag);
  const bool zero = mag == 0 || mag >= QuantOf<T>::kInf;
  const typename QuantOf<T>::Scale s(zero ? 1.0f : QuantOf<T>::value(mag));
  constexpr int kWords = kPer / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
  auto put = [&](int i, u32x4 v) {
    uint32_t w[kWords];
    pack_levels<T>(s, v, w);
    if constexpr (kWords == 1) *reinterpret_cast<uint32_t*>(dst + i * kPer) = zero ? 0u : w[0];
    else *reinterpret_cast<u32x2*>(dst + i * kPer) = zero ? u32x2{0, 0} : u32x2{w[0], w[1]};
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int i = threadIdx.x + h * kQuantThreads;
    if (i < n) put(i, held[h]);
  }
  for (int i = threadIdx.x + kHeld * kQuantThreads; i < n; i += kQuantThreads) put(i, src[i]);
}

// Any columns, stride and alignment, one element at a time.
template <class T>
__global__ __launch_bounds__(kQuantThreads) void k_quantize_any(const T* __restrict__ x, int64_t ldx, int cols,
                                                                int8_t* __restrict__ q, int64_t ldq,
                                                                float* __restrict__ scale) {
  __shared__ uint32_t shared[kQuantThreads / 64];
  const int64_t row = blockIdx.x;
  const T* src = x + row * ldx;
  int8_t* dst = q + row * ldq;
  auto bits = [&](int i) -> uint32_t {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(uint32_t, src[i]);
    else return __builtin_bit_cast(uint16_t, src[i]);
  };
  uint32_t m = 0;
  for (int i = threadIdx.x; i < cols; i += kQuantThreads) m = QuantOf<T>::wider(m, bits(i));
  const uint32_t mag = block_magnitude<T>(m, shared);
  if (threadIdx.x == 0) scale[row] = row_scale<T>(mag);
  const bool zero = mag == 0 || mag >= QuantOf<T>::kInf;
  const typename QuantOf<T>::Scale s(zero ? 1.0f : QuantOf<T>::value(mag));
  for (int i = threadIdx.x; i < cols; i += kQuantThreads)
    dst[i] = zero ? int8_t(0) : static_cast<int8_t>(s.level(QuantOf<T>::value(bits(i))));
}

template <class T>
static void launch_quantize_of(int64_t rows, int64_t cols, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                               float* scale, hipStream_t st) {
  constexpr int kPer = 16 / sizeof(T);
  const bool whole = cols % kPer == 0 && ldx % kPer == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                     ldq % kPer == 0 && reinterpret_cast<uintptr_t>(q) % kPer == 0;
  constexpr int64_t kRowsPerLaunch = int64_t(1) << 23;  // grid x block stays below 2^32 threads
  for (int64_t r = 0; r < rows; r += kRowsPerLaunch)
    hipLaunchKernelGGL(whole ? k_quantize<T> : k_quantize_any<T>,
                       dim3(static_cast<unsigned>(std::min(rows - r, kRowsPerLaunch))), dim3(kQuantThreads), 0, st,
                       static_cast<const T*>(x) + r * ldx, ldx, static_cast<int>(cols), q + r * ldq, ldq, scale + r);
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
// (16-byte aligned, a multiple of 16); the bytes past K are zeroed.
__global__ __launch_bounds__(256) void k_copy_rows(const int8_t* __restrict__ src, int64_t ld, int64_t rows, int K,
                                                   int row16, int8_t* __restrict__ dst, DebugCheck dbg) {
  const int pieces = row16 / 16;
  const int64_t n = rows * pieces;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    const int64_t r = i / pieces;
    const int k0 = static_cast<int>(i - r * pieces) * 16;
    const int8_t* s = src + r * ld + k0;
    u32x4 v{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (k0 + j < K)
        v[j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(dload(dbg, 0, kDbgProjectOperand, s + j))) << (8 * (j % 4));
    dstore(dbg, 1, kDbgProjectWork, reinterpret_cast<u32x4*>(dst + i * 16), v);
  }
}

struct ProjectParams {
  Operand A, B;  // rows of int8 seen as 16-bit pairs: ld and k_lim count pairs
  int32_t K;
  int32_t nk;  // contraction stages of 64 bytes
  const float *a_scale, *b_scale, *bias;
  void* out;
  int64_t ldo, M, N;
  int32_t mblocks, nblocks;
  DebugCheck dbg;  // debug build: span 0 = out, 1 = A, 2 = B, 3 = a_scale, 4 = b_scale, 5 = bias
};

__device__ __forceinline__ void store_as(const DebugCheck& d, float* p, float v) { dstore(d, 0, kDbgProjectOut, p, v); }
__device__ __forceinline__ void store_as(const DebugCheck& d, __bf16* p, float v) {
  dstore(d, 0, kDbgProjectOut, p, static_cast<__bf16>(v));
}
__device__ __forceinline__ void store_as(const DebugCheck& d, _Float16* p, float v) {
  dstore(d, 0, kDbgProjectOut, p, static_cast<_Float16>(v));
}

// Accumulators of one wave of a 256 x 256 int8 block tile: as MainAcc, in
// 32-bit integers.
using IntAcc = i32x4[8][2 * kNBW];

// The bytes of a lane's 16-byte fragment (bytes 16 (lane >> 4) .. + 15 of the
// last 64-byte stage) at and past `valid` cleared.
__device__ __forceinline__ i32x4 keep_bytes(i32x4 v, int valid, int lane) {
  const int left = valid - 16 * (lane >> 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = left - 4 * j;
    v[j] &= n >= 4 ? -1 : n <= 0 ? 0 : (1 << (8 * n)) - 1;
  }
  return v;
}

// acc = A[m0 : m0 + 256] B[n0 : n0 + 256]^T: the ring of LDS stages and the
// schedule of gemm_mainloop (fkl_device.h), each 64-byte stage row holding 64
// int8 instead of 32 bf16, one v_mfma_i32_16x16x64_i8 step per stage. A and B
// fragments use the same assignment of bytes to lanes, so any order of k
// within a stage gives the same sum. In the last stage A's bytes at and past
// K are cleared: what B holds there then does not matter.
__device__ __forceinline__ void int8_mainloop(const Operand& A, const Operand& B, int64_t m0, int64_t n0, int nk,
                                              int last, IntAcc& acc, char* lds) {
  using C = MainCfg;
  constexpr int S = C::kStages;
  constexpr int LA = C::kDmaA;
  constexpr int LB = C::kDmaB;
  constexpr int XA = 8;
  constexpr int XB = 2 * kNBW;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int am = (wave / kWN) * 128;
  const int bn = (wave % kWN) * 64;
  const StageSrc<LA> sa = make_plain_src<kARows, LA>(A, m0, wave, lane);
  const StageSrc<LB> sb = make_plain_src<C::kBExtent, LB>(B, n0, wave, lane);
#pragma unroll
  for (int x = 0; x < XA; ++x)
#pragma unroll
    for (int y = 0; y < XB; ++y) acc[x][y] = i32x4{0, 0, 0, 0};
  block_barrier();
#pragma unroll
  for (int p = 0; p < S; ++p) {
    issue_stage<LA>(sa, p, p < nk, lds + p * C::kStageBytes, wave);
    issue_stage<LB>(sb, p, p < nk, lds + p * C::kStageBytes + kAStageBytes, wave);
  }
  wait_vmcnt<(S - 1) * C::kDmaStage>();
  block_barrier();
  i32x4 a[XA], b[XB];
  auto read = [&](const char* st) {
#pragma unroll
    for (int x = 0; x < XA; ++x) a[x] = __builtin_bit_cast(i32x4, frag_plain(st, am + x * 16, lane));
#pragma unroll
    for (int y = 0; y < XB; ++y) b[y] = __builtin_bit_cast(i32x4, frag_plain(st + kAStageBytes, bn + y * 16, lane));
  };
  auto mma = [&] {
#pragma unroll
    for (int x = 0; x < XA; ++x)
#pragma unroll
      for (int y = 0; y < XB; ++y) acc[x][y] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[x], b[y], acc[x][y], 0, 0, 0);
  };
  read(lds);
  for (int kt = 0; kt + 1 < nk; ++kt) {
    char* cur = lds + (kt % S) * C::kStageBytes;
    const char* nxt = lds + ((kt + 1) % S) * C::kStageBytes;
    mma();
    wait_vmcnt<(S - 2) * C::kDmaStage>();
    block_barrier();
    read(nxt);
    const bool live = kt + S < nk;
    issue_stage<LA>(sa, kt + S, live, cur, wave);
    issue_stage<LB>(sb, kt + S, live, cur + kAStageBytes, wave);
  }
#pragma unroll
  for (int x = 0; x < XA; ++x) a[x] = keep_bytes(a[x], last, lane);
  mma();
  wait_vmcnt<0>();
  block_barrier();
}

// One 256 x 256 output tile per workgroup. MFMA bound.
template <class T>
__global__ __launch_bounds__(kBlockThreads, 1) void k_project(ProjectParams P) {
  __shared__ __align__(16) char lds[kKernelLdsBytes];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wm = wave / kWN;
  const int wn = wave % kWN;
  int mbi, nbi;
  grouped_tile(xcd_contiguous(blockIdx.x, P.mblocks * P.nblocks), P.mblocks, P.nblocks, 8, mbi, nbi);
  const int64_t m0 = static_cast<int64_t>(mbi) * kTile;
  const int64_t n0 = static_cast<int64_t>(nbi) * kTile;
  IntAcc acc;
  dcheck_operand(P.dbg, 1, P.A, m0, kARows, false);
  dcheck_operand(P.dbg, 2, P.B, n0, kTile, false);
  int8_mainloop(P.A, P.B, m0, n0, P.nk, P.K - 64 * (P.nk - 1), acc, lds);
  // Epilogue: each 256 x 128 half tile of sums staged in LDS, then scaled and
  // stored with 32 lanes on 128 consecutive columns.
  int32_t* stage = reinterpret_cast<int32_t*>(lds);
  const int rmax = static_cast<int>(min<int64_t>(kTile, P.M - m0));
  for (int half = 0; half < 2; ++half) {
    const int64_t cbase = n0 + half * 128;
    const int cmax = static_cast<int>(min<int64_t>(128, P.N - cbase));
    const int c4 = (tid & 31) * 4;
    float sb[4], bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = c4 + j < cmax;
      sb[j] = in ? dload(P.dbg, 4, kDbgProjectOperand, P.b_scale + cbase + c4 + j) : 0.0f;
      bias[j] = in && P.bias ? dload(P.dbg, 5, kDbgProjectOperand, P.bias + cbase + c4 + j) : 0.0f;
    }
    if ((wn >> 1) == half) {
      const int cw = (wn & 1) * 64;
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int y = 0; y < 2 * kNBW; ++y)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            stage[(wm * 128 + acc_row(x, i, lane)) * kStageLd + cw + acc_col(y, lane)] = acc[x][y][i];
    }
    __syncthreads();
    for (int r = tid >> 5; r < rmax; r += kBlockThreads / 32) {
      const float sa = dload(P.dbg, 3, kDbgProjectOperand, P.a_scale + m0 + r);
      const i32x4 v = *reinterpret_cast<const i32x4*>(stage + r * kStageLd + c4);
      T* o = static_cast<T*>(P.out) + (m0 + r) * P.ldo + cbase + c4;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c4 + j < cmax) store_as(P.dbg, o + j, fmaf(static_cast<float>(v[j]) * sa, sb[j], bias[j]));
    }
    __syncthreads();
  }
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
    const hipError_t e = launch_quantize(p.M, p.K, p.a_type, g.a, p.lda, q, row16, s, st);
    if (e != hipSuccess) return e;
    a = q, lda = row16, a_scale = s;
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
  P.nk = static_cast<int32_t>(ceil_div(p.K, 64));
  P.a_scale = a_scale, P.b_scale = g.b_scale, P.bias = g.bias;
  P.out = g.out;
  P.ldo = p.ldo, P.M = p.M, P.N = p.N;
  P.mblocks = static_cast<int32_t>(ceil_div(p.M, kTile));
  P.nblocks = static_cast<int32_t>(ceil_div(p.N, kTile));
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
  TraceScope ts(st, "project", flops, bytes);
  auto* k = p.out_type == FKL_F32 ? k_project<float> : p.out_type == FKL_BF16 ? k_project<__bf16> : k_project<_Float16>;
  hipLaunchKernelGGL(k, dim3(static_cast<unsigned>(P.mblocks) * P.nblocks), dim3(kBlockThreads), 0, st, P);
  return hipGetLastError();
}

}  // namespace fkl
