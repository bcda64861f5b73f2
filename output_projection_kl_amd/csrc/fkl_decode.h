// Host-side plans and kernel launchers of the 8-bit head (fkl_quantize,
// fkl_project) and of sampling (fkl_sample). Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fkl.h"
#include "fkl_internal.h"

namespace fkl {

inline int type_bytes(int type) { return type == FKL_F32 ? 4 : type == FKL_I8 ? 1 : 2; }

// Products of rows of up to this many 8-bit values cannot overflow a 32-bit
// sum: 128 * 128 * K < 2^31.
constexpr int64_t kProjectMaxK = 131071;

// Debug build: access classes of these kernels, bits of the call's violation
// word (at kDebugWordOffset in the workspace's first 256 bytes).
enum DecodeDebugBit : uint32_t {
  kDbgProjectOperand = 1u << 0,  // a, b, their packed copies, scales and bias
  kDbgProjectOut = 1u << 1,      // the product
  kDbgProjectWork = 1u << 2,     // the workspace: quantised or packed operands, partial sums
  kDbgSampleLogits = 1u << 3,    // logits, ids, random numbers and per-row settings
  kDbgSampleOut = 1u << 4,       // tokens and log-probabilities
  kDbgSampleWork = 1u << 5,      // the workspace: per-row statistics
};
constexpr int kDecodeDebugBits = 6;

constexpr int64_t kLastLevelBytes = int64_t(256) << 20;  // of cache between the L2s and memory

// How the product is laid out on the GPU: the split-contraction kernel for few
// output elements, or block tiles.
enum ProjectShapeId {
  kProjectSkinny,
  kProject16x64,
  kProject32x64,
  kProject64,
  kProject64x128,
  kProject128,
  kProject128x256,
  kProject256x128,
  kProject256
};

// How the block tiles read B. Once: with the hint that nothing else will ask
// for it; by lines: each row in whole cache lines although it does not start
// at one (for tiles of up to kProjectLinesRows rows).
enum ProjectRead { kReadPlain, kReadOnce, kReadOnceByLines };
constexpr int kProjectLinesRows = 32;

struct ProjectPlan {
  int64_t M, N, K, lda, ldb, ldo;
  int a_type, out_type;
  int64_t row_a;            // bytes of a quantised row of a in the workspace
  bool once;                // every byte of b is read once, and b is larger than the last-level cache
  bool a_copied, b_copied;  // the 8-bit operand is copied to rows of round_up(K, 16) bytes
  ProjectShapeId shape;
  int splits;       // of the contraction, each of k_split bytes (1: none)
  int64_t k_split;
  // workspace offsets (bytes): the quantised or copied a, its scales, the copied b, the splits' sums
  size_t off_a, off_a_scale, off_b, off_sums, bytes;
};

struct ProjectArgs {
  const void* a;
  const float* a_scale;
  const int8_t* b;
  const float* b_scale;
  const float* bias;
  void* out;
  char* ws;
};

enum SampleRoute { kSampleShort, kSampleRow, kSampleScan, kSampleLong };

struct SamplePlan {
  int64_t N, V, ld, ld_ids;
  int type;
  SampleRoute route;
  // the scan: groups of 2^group_shift elements and chunks of chunk_elems per
  // row, counted with the up to 7 elements between a 16-byte boundary and the
  // row's start
  int64_t groups, chunks, chunk_elems;
  int group_shift;
  size_t off_group_max, off_chunk_max, off_chunk_mass, off_chunk_hist, bytes;
};

constexpr int64_t kSampleShortMaxV = 1024;
constexpr int64_t kSampleScanMaxV = (int64_t(1) << 20) - 8;
constexpr int64_t kSampleRowMax = 8192;
constexpr int64_t kSampleMaxGroups = 4160;  // a little over 2^18 / 64: rows of 2^18 entries at any alignment
constexpr int64_t kSampleMaxChunks = 64;
constexpr int64_t kSampleChunk = 4096;  // elements per scan workgroup, or twice or four times as many
constexpr int64_t kSampleHistBytes = 512 * 8;  // one chunk's mass histogram

struct SampleArgs {
  const void* logits;
  const int32_t* ids;
  const float* u;
  fkl_sample_params params;
  int32_t* token;
  float* logprob;
  char* ws;
};

fkl_status make_project_plan(const fkl_project_shape* s, ProjectPlan* p);
fkl_status make_sample_plan(const fkl_sample_shape* s, SamplePlan* p);

hipError_t launch_quantize(int64_t rows, int64_t cols, int type, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                           float* scale, hipStream_t stream);
hipError_t launch_project(const ProjectPlan& p, const ProjectArgs& a, hipStream_t stream);
hipError_t launch_sample(const SamplePlan& p, const SampleArgs& a, hipStream_t stream);

}  // namespace fkl
