// C ABI of the 8-bit head and of sampling: argument checks (pure host code,
// no HIP call before they pass), workspace plans, dispatch to the launchers in
// fkl_int8.hip and fkl_sample.hip.
#include <algorithm>
#include <cmath>
#include <string>

#include "fkl.h"
#include "fkl_decode.h"
#include "fkl_internal.h"

namespace {

using fkl::set_error;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Row strides of 8-bit operands that the kernels read directly: whole 16-byte
// pieces, and a tile's 256 rows within a 32-bit buffer size.
bool readable_stride(int64_t ld) { return ld % 16 == 0 && ld <= (int64_t(1) << 22); }

bool is_float_type(int t) { return t == FKL_F32 || t == FKL_BF16 || t == FKL_F16; }

// The debug build keeps its violation word at the start of every workspace.
#ifdef FKL_DEBUG
constexpr size_t kControlBytes = 256;
#else
constexpr size_t kControlBytes = 0;
#endif

fkl_status check_workspace(const void* workspace, size_t given, size_t need, const char* size_call) {
  if (need == 0) return FKL_OK;
  if (!workspace) return set_error(FKL_EWORKSPACE, "workspace is NULL");
  if (!aligned(workspace, 256)) return set_error(FKL_EWORKSPACE, "workspace must be 256-byte aligned");
  if (given < need) return set_error(FKL_EWORKSPACE, std::string("workspace is smaller than ") + size_call);
  return FKL_OK;
}

fkl_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return FKL_OK;
  return set_error(FKL_EDEVICE, std::string(what) + " launch failed: " + hipGetErrorString(e));
}

// Debug build (FKL_DEBUG): the violation word of a call is cleared before its
// first launch; after its last the host waits and reports what fired.
fkl_status debug_begin(char* ws, hipStream_t stream) {
#ifdef FKL_DEBUG
  return launched(fkl::launch_debug_clear(reinterpret_cast<uint32_t*>(ws + fkl::kDebugWordOffset), stream),
                  "debug word clear");
#else
  (void)ws, (void)stream;
  return FKL_OK;
#endif
}

fkl_status debug_end(char* ws, hipStream_t stream) {
#ifdef FKL_DEBUG
  static const char* const kNames[fkl::kDecodeDebugBits] = {"project operands", "project output",
                                                            "project workspace", "sample inputs",
                                                            "sample outputs",    "sample workspace"};
  uint32_t host = 0;
  hipError_t e = hipMemcpyAsync(&host, ws + fkl::kDebugWordOffset, sizeof(host), hipMemcpyDeviceToHost, stream);
  if (e == hipSuccess) e = hipStreamSynchronize(stream);
  if (e != hipSuccess) return launched(e, "debug word read");
  if (host != 0) {
    std::string msg = "device bounds check failed (accesses skipped):";
    for (int b = 0; b < fkl::kDecodeDebugBits; ++b)
      if (host & (1u << b)) msg += std::string(" ") + kNames[b] + ";";
    return set_error(FKL_EDEVICE, msg);
  }
#else
  (void)ws, (void)stream;
#endif
  return FKL_OK;
}

}  // namespace

namespace fkl {

// The layout of the product.
//
// A b larger than the last-level cache is not there at the next call. For up
// to 256 rows it is read once, memory decides, and its loads say so (they are
// non-temporal): 128256 x 4096 rows, 85 instead of 99 us for 8 rows of a, 91
// instead of 105 for 30, 111 instead of 120 for 64, 149 instead of 155 for 200.
// A b that the cache could hold is better kept there: 32000 x 4096, the same at
// every call, took 30 us with the hint and 23 without. Rows that do not start
// at cache lines share lines, which the hint lets go in between: such rows are
// read by whole lines (up to 32 rows of a: 201088 x 2880, 101 instead of 115 us
// for 16, 111 instead of 122 for 32), or without the hint (48: 129 us, 134 by
// whole lines, 144 with the hint alone).
//
// Otherwise the layout with the least estimated time, us. A block tile's stage (128
// bytes of the contraction) takes `filled` of a CU that as many workgroups
// share as fit, and `alone` for a workgroup with a CU to itself, whichever is
// longer over the rounds that the tiles take; then the tile is stored. The
// constants are fitted to the times of the layouts at 157 sizes (M 1 to 8192,
// N 64 to 201088, K 64 to 8192): the layout that they pick took 1.5% longer
// than the fastest one in the mean. Both sides at some of them: 8192 x 8192 x
// 4096 (M, N, K): 232 us as 256 x 256, 292 as 128 x 256, 328 as 128 x 128; 2048
// x 4096 x 4096: 51, 39 and 44; 201 x 32003 x 2887: 50, 36 and 41; 48 x 32000 x
// 4096: 37 as 64 x 128, 36 as 64 x 64; 32 x 32000 x 4096: 34 as 32 x 64, 37 as
// 16 x 64; 5 x 1024 x 1024: 6.1 as 16 x 16, 7.3 as 16 x 64; 1 x 128 x 5120:
// 8.7 as 16 x 16, 19.7 as 64 x 64, 10.8 of those with the contraction split.
static void choose_project_shape(ProjectPlan* p) {
  struct Tile {
    ProjectShapeId id;
    int tm, tn, per_cu;
    double alone, filled;
  };
  static const Tile kTiles[] = {
      {kProject16x64, 16, 64, 3, 0.21, 0.16},   {kProject32x64, 32, 64, 3, 0.24, 0.19},
      {kProject64, 64, 64, 3, 0.28, 0.26},      {kProject64x128, 64, 128, 2, 0.80, 0.50},
      {kProject128, 128, 128, 2, 0.85, 0.68},   {kProject128x256, 128, 256, 1, 0.75, 1.20},
      {kProject256x128, 256, 128, 1, 0.76, 1.10}, {kProject256, 256, 256, 1, 1.07, 1.80},
  };
  p->splits = 1;
  p->k_split = p->K;
  p->once = p->M <= 256 && p->N * (p->b_copied ? round_up(p->K, 16) : p->ldb) > kLastLevelBytes;
  if (p->once) {
    p->shape = p->M <= 16 ? kProject16x64 : p->M <= 32 ? kProject32x64 : p->M <= 64 ? kProject64x128
             : p->M <= 128 ? kProject128x256 : kProject256;
    return;
  }
  const double kLaunch = 2.4;  // a launch's own time
  const double kJoin = 4.2;    // the second launch of a split contraction
  const double m = static_cast<double>(p->M), n = static_cast<double>(p->N), k = static_cast<double>(p->K);
  const double memory = (n * k + m * k + m * n * type_bytes(p->out_type)) / 6.5e6;
  const int64_t stages = ceil_div(p->K, 128);
  // 16 x 16 tiles, two workgroups a CU: one tile's latency, then less for each
  // further one; B is read again for every 16 rows
  const int64_t small = ceil_div(p->M, 16) * ceil_div(p->N, 16);
  p->shape = kProjectSkinny;
  double best = kLaunch + 0.95 * k / 1024 + static_cast<double>(ceil_div(small, 512) - 1) * (0.29 * k / 1024 + 0.3);
  best = std::max(best, static_cast<double>(ceil_div(p->M, 16)) * n * k / 3.6e6);
  for (const Tile& t : kTiles) {
    const int64_t tiles = ceil_div(p->M, t.tm) * ceil_div(p->N, t.tn);
    const double rounds = static_cast<double>(ceil_div(tiles, int64_t(kTargetBlocks) * t.per_cu));
    const double per_cu = static_cast<double>(tiles) / kTargetBlocks;
    const double sums = static_cast<double>(stages) * std::max(t.alone * rounds, t.filled * per_cu);
    const double store = 4.0 * t.tm * t.tn / 65536 * std::max(rounds, per_cu) * type_bytes(p->out_type) / 2;
    // rows past M are computed in vain: a little even where memory decides
    const double est = std::max(kLaunch + sums + store, memory) + 0.02 * sums;
    if (est < best) best = est, p->shape = t.id;
  }
  // 64 x 64 tiles with the contraction split over more workgroups and the sums
  // joined by a second launch: for long contractions of few tiles
  const int64_t tiles = ceil_div(p->M, 64) * ceil_div(p->N, 64);
  for (int64_t splits = 2; splits <= 32 && splits <= stages / 2 && tiles * splits <= 3 * kTargetBlocks; splits *= 2) {
    const int64_t per = ceil_div(stages, splits);
    const double one = std::max(0.28, 0.26 * static_cast<double>(tiles * splits) / kTargetBlocks);
    const double est = 2 * kLaunch + kJoin + static_cast<double>(per) * one + static_cast<double>(splits) * m * n * 2e-6;
    if (est < best) {
      best = est, p->shape = kProject64;
      p->k_split = per * 128;
      p->splits = static_cast<int>(ceil_div(p->K, p->k_split));
    }
  }
}

fkl_status make_project_plan(const fkl_project_shape* s, ProjectPlan* p) {
  if (!s) return set_error(FKL_EINVAL, "shape is NULL");
  if (s->M < 0) return set_error(FKL_EINVAL, "M must be >= 0");
  if (s->N < 1 || s->K < 1) return set_error(FKL_EINVAL, "N and K must be >= 1");
  const int64_t kMax = (int64_t(1) << 31) - 1024;
  if (s->M > kMax || s->N > kMax) return set_error(FKL_EUNSUPPORTED, "M and N must be < 2^31 - 1024");
  if (s->K > kProjectMaxK)
    return set_error(FKL_EUNSUPPORTED, "K must be <= 131071 (a 32-bit sum of 8-bit products could overflow)");
  if (s->a_type != FKL_I8 && !is_float_type(s->a_type))
    return set_error(FKL_EINVAL, "a_type must be FKL_I8, FKL_F32, FKL_BF16 or FKL_F16");
  if (!is_float_type(s->out_type)) return set_error(FKL_EINVAL, "out_type must be FKL_F32, FKL_BF16 or FKL_F16");
  if (s->lda < s->K || s->ldb < s->K) return set_error(FKL_EINVAL, "lda and ldb must be >= K");
  if (s->ldo < s->N) return set_error(FKL_EINVAL, "ldo must be >= N");
  const int64_t kMaxLd = int64_t(1) << 40;
  if (s->lda > kMaxLd || s->ldb > kMaxLd || s->ldo > kMaxLd)
    return set_error(FKL_EUNSUPPORTED, "lda, ldb and ldo must be <= 2^40");
  if (s->flags & ~static_cast<uint32_t>(FKL_PROJECT_COPY_A | FKL_PROJECT_COPY_B))
    return set_error(FKL_EINVAL, "unknown fkl_project_shape flag");
  if (ceil_div(s->M, kTile) * ceil_div(s->N, kTile) >= (int64_t(1) << 22))
    return set_error(FKL_EUNSUPPORTED, "out must hold fewer than 2^22 tiles of 256 x 256");
  p->M = s->M, p->N = s->N, p->K = s->K;
  p->lda = s->lda, p->ldb = s->ldb, p->ldo = s->ldo;
  p->a_type = s->a_type, p->out_type = s->out_type;
  p->a_copied = s->a_type == FKL_I8 && ((s->flags & FKL_PROJECT_COPY_A) || !readable_stride(s->lda));
  p->b_copied = (s->flags & FKL_PROJECT_COPY_B) || !readable_stride(s->ldb);
  const size_t row = static_cast<size_t>(round_up(s->K, 16));
  size_t off = kControlBytes;
  p->off_a = off;
  // a quantised a in rows that start at cache lines
  p->row_a = round_up(s->K, s->a_type != FKL_I8 ? 128 : 16);
  if (p->a_copied || s->a_type != FKL_I8) off = align256(off + static_cast<size_t>(s->M * p->row_a));
  p->off_a_scale = off;
  if (s->a_type != FKL_I8) off = align256(off + static_cast<size_t>(s->M) * 4);
  p->off_b = off;
  if (p->b_copied) off = align256(off + static_cast<size_t>(s->N) * row);
  choose_project_shape(p);
  p->off_sums = off;
  if (p->splits > 1)
    off = align256(off + static_cast<size_t>(p->splits) * s->M * static_cast<size_t>(round_up(s->N, 4)) * 4);
  p->bytes = off;
  return FKL_OK;
}

fkl_status make_sample_plan(const fkl_sample_shape* s, SamplePlan* p) {
  if (!s) return set_error(FKL_EINVAL, "shape is NULL");
  if (s->N < 0) return set_error(FKL_EINVAL, "N must be >= 0");
  if (s->V < 1) return set_error(FKL_EINVAL, "V must be >= 1");
  const int64_t kMax = (int64_t(1) << 31) - 1024;
  if (s->N > kMax || s->V > kMax) return set_error(FKL_EUNSUPPORTED, "N and V must be < 2^31 - 1024");
  if (!is_float_type(s->type)) return set_error(FKL_EINVAL, "type must be FKL_F32, FKL_BF16 or FKL_F16");
  if (s->ld < s->V) return set_error(FKL_EINVAL, "ld must be >= V");
  if (s->ld_ids < 0) return set_error(FKL_EINVAL, "ld_ids must be >= 0");
  const int64_t kMaxLd = int64_t(1) << 40;
  if (s->ld > kMaxLd || s->ld_ids > kMaxLd) return set_error(FKL_EUNSUPPORTED, "ld and ld_ids must be <= 2^40");
  p->N = s->N, p->V = s->V, p->ld = s->ld, p->ld_ids = s->ld_ids;
  p->type = s->type;
  // Short rows, up to one per CU, take one launch for the scan and the pick: a
  // call of 64 x 8000 fp32 with top-k 50 and top-p, or with min-p, 11.3 instead
  // of 13.4 us, most of either the host's. Longer rows lose more by a draw
  // from the whole row than the launch costs (64 x 16000 without filters: 17
  // instead of 14).
  p->route = s->V <= kSampleShortMaxV                                                  ? kSampleShort
             : s->V + 7 <= kSampleRowMax && s->N <= static_cast<int64_t>(kTargetBlocks) ? kSampleRow
             : s->V <= kSampleScanMaxV                                                 ? kSampleScan
                                                                                       : kSampleLong;
  p->groups = p->chunks = p->chunk_elems = p->group_shift = 0;
  size_t off = kControlBytes;
  p->off_group_max = p->off_chunk_max = p->off_chunk_mass = p->off_chunk_hist = off;
  if (p->route == kSampleRow || p->route == kSampleScan) {
    // Chunks of 4096 entries, a workgroup of 256 threads each: the draw reads
    // one, and small workgroups share the CUs evenly (130 x 50257 fp16 without
    // filters: 12 us for the scan and 9 for the pick, 17 and 14 with chunks of
    // 16384). Long rows add up their chunks' histograms: twice the chunk where
    // that leaves two workgroups per CU (64 x 128256 bf16, top-p: 14.5 and 29.5
    // us, 16 and 31 with 4096; 512 x 201088 fp32: 117 and 56, 122 and 67). The
    // longest need the largest to have no more than 64.
    p->chunk_elems = kSampleChunk;
    if (p->route == kSampleRow || s->V + 7 > kSampleMaxChunks * 2 * kSampleChunk) p->chunk_elems = 4 * kSampleChunk;
    else if (s->V + 7 > kSampleMaxChunks * kSampleChunk ||
             (s->V > 65536 && s->N * ceil_div(s->V, 2 * kSampleChunk) >= 2 * kTargetBlocks))
      p->chunk_elems = 2 * kSampleChunk;
    // the smallest groups of which a row has few enough: top-k's bound, the
    // k-th largest group maximum, needs many more groups than k
    p->group_shift = s->V + 7 <= 4096 * 16 ? 4 : s->V + 7 <= kSampleMaxGroups * 64 ? 6 : 8;
    p->groups = ceil_div(s->V + 7, int64_t(1) << p->group_shift);
    p->chunks = ceil_div(s->V + 7, p->chunk_elems);
    const size_t n = static_cast<size_t>(s->N);
    off = align256(off + n * p->groups * 4);
    p->off_chunk_max = off;
    off = align256(off + n * p->chunks * 4);
    p->off_chunk_mass = off;
    off = align256(off + n * p->chunks * 8);
    p->off_chunk_hist = off;
    off = align256(off + n * p->chunks * kSampleHistBytes);
  }
  p->bytes = off;
  return FKL_OK;
}

}  // namespace fkl

extern "C" {

fkl_status fkl_quantize(int64_t rows, int64_t cols, int32_t type, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                        float* scale, void* stream) {
  if (rows < 0) return set_error(FKL_EINVAL, "rows must be >= 0");
  if (cols < 1) return set_error(FKL_EINVAL, "cols must be >= 1");
  const int64_t kMax = (int64_t(1) << 31) - 1024;
  if (rows > kMax || cols > kMax) return set_error(FKL_EUNSUPPORTED, "rows and cols must be < 2^31 - 1024");
  if (!is_float_type(type)) return set_error(FKL_EINVAL, "type must be FKL_F32, FKL_BF16 or FKL_F16");
  if (ldx < cols || ldq < cols) return set_error(FKL_EINVAL, "ldx and ldq must be >= cols");
  const int64_t kMaxLd = int64_t(1) << 40;
  if (ldx > kMaxLd || ldq > kMaxLd) return set_error(FKL_EUNSUPPORTED, "ldx and ldq must be <= 2^40");
  if (rows == 0) return FKL_OK;
  if (!x || !q || !scale) return set_error(FKL_EINVAL, "x, q and scale must not be NULL");
  if (!aligned(x, fkl::type_bytes(type)) || !aligned(scale, 4))
    return set_error(FKL_EINVAL, "x must be aligned to its type and scale to 4 bytes");
  return launched(fkl::launch_quantize(rows, cols, type, x, ldx, q, ldq, scale, static_cast<hipStream_t>(stream)),
                  "quantize");
}

fkl_status fkl_project_workspace_size(const fkl_project_shape* shape, size_t* bytes) {
  fkl::ProjectPlan p;
  const fkl_status st = fkl::make_project_plan(shape, &p);
  if (st != FKL_OK) return st;
  if (bytes) *bytes = p.bytes;
  return FKL_OK;
}

fkl_status fkl_project(const fkl_project_shape* shape, const void* a, const float* a_scale, const int8_t* b,
                       const float* b_scale, const float* bias, void* out, void* workspace, size_t workspace_bytes,
                       void* stream) {
  fkl::ProjectPlan p;
  fkl_status st = fkl::make_project_plan(shape, &p);
  if (st != FKL_OK) return st;
  if (p.M == 0) return FKL_OK;
  if (!a || !b || !b_scale || !out) return set_error(FKL_EINVAL, "a, b, b_scale and out must not be NULL");
  if (p.a_type == FKL_I8 && !a_scale) return set_error(FKL_EINVAL, "a_scale must not be NULL with 8-bit rows");
  if (p.a_type != FKL_I8 && a_scale)
    return set_error(FKL_EINVAL, "a_scale must be NULL with floating rows: they are quantised by the call");
  if (!aligned(a, fkl::type_bytes(p.a_type)) || !aligned(out, fkl::type_bytes(p.out_type)))
    return set_error(FKL_EINVAL, "a and out must be aligned to their types");
  if ((p.a_type == FKL_I8 && !p.a_copied && !aligned(a, 16)) || (!p.b_copied && !aligned(b, 16)))
    return set_error(FKL_EINVAL, "an 8-bit operand that is read where it is must be 16-byte aligned "
                                 "(FKL_PROJECT_COPY_A and FKL_PROJECT_COPY_B copy it first)");
  if ((a_scale && !aligned(a_scale, 4)) || !aligned(b_scale, 4) || (bias && !aligned(bias, 4)))
    return set_error(FKL_EINVAL, "a_scale, b_scale and bias must be 4-byte aligned");
  st = check_workspace(workspace, workspace_bytes, p.bytes, "fkl_project_workspace_size()");
  if (st != FKL_OK) return st;
  char* ws = static_cast<char*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  st = debug_begin(ws, s);
  if (st != FKL_OK) return st;
  const fkl::ProjectArgs args{a, a_scale, b, b_scale, bias, out, ws};
  st = launched(fkl::launch_project(p, args, s), "project");
  if (st != FKL_OK) return st;
  return debug_end(ws, s);
}

fkl_status fkl_sample_workspace_size(const fkl_sample_shape* shape, size_t* bytes) {
  fkl::SamplePlan p;
  const fkl_status st = fkl::make_sample_plan(shape, &p);
  if (st != FKL_OK) return st;
  if (bytes) *bytes = p.bytes;
  return FKL_OK;
}

fkl_status fkl_sample(const fkl_sample_shape* shape, const fkl_sample_params* params, const void* logits,
                      const int32_t* ids, const float* u, int32_t* token, float* logprob, void* workspace,
                      size_t workspace_bytes, void* stream) {
  fkl::SamplePlan p;
  fkl_status st = fkl::make_sample_plan(shape, &p);
  if (st != FKL_OK) return st;
  if (!params) return set_error(FKL_EINVAL, "params is NULL");
  if (!params->temperature_rows && !(params->temperature >= 0.0f && std::isfinite(params->temperature)))
    return set_error(FKL_EINVAL, "temperature must be finite and >= 0");
  if (!params->top_p_rows && std::isnan(params->top_p)) return set_error(FKL_EINVAL, "top_p must not be NaN");
  if (!params->min_p_rows && std::isnan(params->min_p)) return set_error(FKL_EINVAL, "min_p must not be NaN");
  if (!aligned(params->temperature_rows, 4) || !aligned(params->top_k_rows, 4) || !aligned(params->top_p_rows, 4) ||
      !aligned(params->min_p_rows, 4))
    return set_error(FKL_EINVAL, "the per-row settings must be 4-byte aligned");
  if (p.N == 0) return FKL_OK;
  if (!logits || !u || !token) return set_error(FKL_EINVAL, "logits, u and token must not be NULL");
  if (ids && p.ld_ids < p.V) return set_error(FKL_EINVAL, "ld_ids must be >= V");
  if (!aligned(logits, fkl::type_bytes(p.type)) || !aligned(ids, 4) || !aligned(u, 4) || !aligned(token, 4) ||
      !aligned(logprob, 4))
    return set_error(FKL_EINVAL, "logits must be aligned to their type; ids, u, token and logprob to 4 bytes");
  st = check_workspace(workspace, workspace_bytes, p.bytes, "fkl_sample_workspace_size()");
  if (st != FKL_OK) return st;
  char* ws = static_cast<char*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  st = debug_begin(ws, s);
  if (st != FKL_OK) return st;
  const fkl::SampleArgs args{logits, ids, u, *params, token, logprob, ws};
  st = launched(fkl::launch_sample(p, args, s), "sample");
  if (st != FKL_OK) return st;
  return debug_end(ws, s);
}

}  // extern "C"
