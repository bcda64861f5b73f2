// Host-only check of csrc/fkl_decode_api.cpp, built with g++ under
// AddressSanitizer and UndefinedBehaviorSanitizer, no GPU and no HIP runtime.
// The launchers are stubs that check the plan they are handed: every
// workspace region inside the workspace, aligned and disjoint, operands within
// what the kernels' 32-bit buffer descriptors and grids address. main() drives
// the entry points over edge shapes and a seeded random sweep.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <string>

#include "fkl_decode.h"

namespace {
int g_fail = 0;
long g_launches = 0;
size_t g_given = 0;
#define CHECK(cond)                                                           \
  do {                                                                        \
    if (!(cond)) {                                                            \
      std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      ++g_fail;                                                               \
    }                                                                         \
  } while (0)
}  // namespace

extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }

namespace fkl {

fkl_status set_error(fkl_status st, const std::string& msg) {
  CHECK(!msg.empty());
  return st;
}

hipError_t launch_quantize(int64_t rows, int64_t cols, int type, const void*, int64_t ldx, int8_t*, int64_t ldq, float*,
                           hipStream_t) {
  ++g_launches;
  CHECK(rows > 0 && cols > 0 && cols < INT32_MAX && type != FKL_I8 && ldx >= cols && ldq >= cols);
  return hipSuccess;
}

hipError_t launch_project(const ProjectPlan& p, const ProjectArgs& a, hipStream_t) {
  ++g_launches;
  CHECK(p.bytes <= g_given && p.M > 0 && p.K <= kProjectMaxK);
  const size_t row = static_cast<size_t>(round_up(p.K, 16));
  size_t end = 0;
  CHECK(p.off_a >= end && p.off_a % 256 == 0);
  if (p.a_type != FKL_I8 || p.a_copied) end = p.off_a + p.M * row;
  CHECK(p.off_a_scale >= end && p.off_a_scale % 256 == 0);
  if (p.a_type != FKL_I8) end = p.off_a_scale + p.M * 4;
  CHECK(p.off_b >= end && p.off_b % 256 == 0);
  if (p.b_copied) end = p.off_b + p.N * row;
  CHECK(p.off_sums >= end && p.off_sums % 256 == 0);
  CHECK(p.splits >= 1 && p.splits <= 32 && p.splits * p.k_split >= p.K);
  if (p.splits > 1) {  // every split has something to add up, in whole stages
    CHECK(p.shape == kProject64 && p.k_split % 128 == 0 && (p.splits - 1) * p.k_split < p.K);
    end = p.off_sums + static_cast<size_t>(p.splits) * p.M * round_up(p.N, 4) * 4;
  }
  CHECK(p.bytes >= end);
  if (p.a_type == FKL_I8 && !p.a_copied) CHECK(p.lda % 16 == 0 && kTile * p.lda <= INT32_MAX);
  if (!p.b_copied) CHECK(p.ldb % 16 == 0 && kTile * p.ldb <= INT32_MAX);
  CHECK(ceil_div(p.M, kTile) * ceil_div(p.N, kTile) * 512 < (int64_t(1) << 32));
  CHECK((a.a_scale != nullptr) == (p.a_type == FKL_I8));
  return hipSuccess;
}

hipError_t launch_sample(const SamplePlan& p, const SampleArgs& a, hipStream_t) {
  ++g_launches;
  CHECK(p.bytes <= g_given && p.N > 0 && p.V > 0 && p.ld >= p.V && (!a.ids || p.ld_ids >= p.V));
  return hipSuccess;
}

}  // namespace fkl

int main() {
  std::mt19937_64 rng(3);
  auto upto = [&](int64_t n) { return static_cast<int64_t>(rng() % static_cast<uint64_t>(n)) + 1; };
  char* const at = reinterpret_cast<char*>(uintptr_t(1) << 20);
  for (int i = 0; i < 20000; ++i) {
    const int64_t big = i % 7 == 0 ? 3000000000ll : i % 3 == 0 ? 200000 : 500;
    fkl_project_shape s{upto(big) - 1, upto(big), upto(i % 5 ? 9000 : 140000), 0, 0, 0, static_cast<int32_t>(rng() % 4),
                        static_cast<int32_t>(rng() % 3), static_cast<uint32_t>(rng() % 4)};
    auto stride = [&](int64_t n) { return rng() % 2 ? fkl::round_up(n, 16) : n + upto(40) - 1; };
    s.lda = stride(s.K), s.ldb = i % 11 ? stride(s.K) : (int64_t(1) << 22) + 16 * upto(3), s.ldo = stride(s.N);
    size_t need = 0;
    fkl_status st = fkl_project_workspace_size(&s, &need);
    CHECK(st == FKL_OK || st == FKL_EUNSUPPORTED);
    if (st != FKL_OK) continue;
    const float* scale = s.a_type == FKL_I8 ? reinterpret_cast<float*>(at) : nullptr;
    auto call = [&](size_t bytes) {
      g_given = bytes;
      return fkl_project(&s, at, scale, reinterpret_cast<int8_t*>(at), reinterpret_cast<float*>(at), nullptr, at, at,
                         bytes, nullptr);
    };
    CHECK(call(need) == FKL_OK);
    if (s.M > 0 && need > 0) CHECK(call(need - 1) == FKL_EWORKSPACE);
    fkl_sample_shape v{s.M, s.N, s.ldo, s.ldo, static_cast<int32_t>(rng() % 3)};
    const fkl_sample_params pr{nullptr, nullptr, nullptr, nullptr, 1.0f, 0, 1.0f, 0.0f};
    CHECK(fkl_sample_workspace_size(&v, &need) == FKL_OK);
    g_given = need;
    CHECK(fkl_sample(&v, &pr, at, reinterpret_cast<int32_t*>(at), reinterpret_cast<float*>(at),
                     reinterpret_cast<int32_t*>(at), reinterpret_cast<float*>(at), at, need, nullptr) == FKL_OK);
  }
  std::printf("launches %ld failures %d\n", g_launches, g_fail);
  return g_fail != 0;
}
