// Host-side exerciser of the root-mean-square norm, 8-bit product and beam search entry points,
// built with AddressSanitizer and UndefinedBehaviorSanitizer (tests/test_host_sanitizers_serve.py).
// As host_sanitizer_ops_driver.cpp: extreme and inconsistent sizes, NULL and misaligned fake
// pointers, where no GPU is visible, so that a call which passes validation stops at the device
// check. Every call must return a documented code other than LCE_OK (size queries, and a reordering
// of nothing: a documented code).
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>
#include <vector>

#include "lce_masked.h"

extern "C" int hipGetDeviceCount(int* count);  // the runtime's int-sized hipError_t

namespace {

int failures = 0;
long calls = 0;

void expect(int rc, const char* what, bool query = false) {
  ++calls;
  if (rc < LCE_OK || rc > LCE_ERR_BAD_DTYPE || (rc == LCE_OK && !query)) {
    std::fprintf(stderr, "%s: status %d\n", what, rc);
    ++failures;
  }
}

const int64_t kMax = std::numeric_limits<int64_t>::max();
const int64_t kMin = std::numeric_limits<int64_t>::min();
const int64_t kSizes[] = {kMin, -1, 0, 1, 16, 1024, int64_t(1) << 20, (int64_t(1) << 23) + 1,
                          (int64_t(1) << 31) - 1, int64_t(1) << 31, int64_t(1) << 62, kMax};
const int64_t kFew[] = {-1, 0, 1, 16, 64, 4096, int64_t(1) << 20, (int64_t(1) << 31) - 1, kMax};

alignas(256) unsigned char arena[1 << 17];
void* fake(int i) { return arena + 4096 * (i % 32); }
template <class T>
T* at(int i) {
  return static_cast<T*>(fake(i));
}

}  // namespace

int main() {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == 0 && ndev > 0) {
    std::printf("skipped: a GPU is visible\n");
    return 0;
  }
  const size_t big = size_t(1) << 60;
  size_t bytes = 0;
  for (int64_t n : kSizes)
    for (int64_t h : kSizes) {
      expect(rmsnorm_workspace_size(n, h, &bytes), "norm ws", true);
      for (int64_t ld : kSizes)
        for (int dt : {-1, 0, 1, 2, 3})
          for (float eps : {1e-6f, -1.f}) {
            expect(rmsnorm_fwd(fake(0), dt, n, h, ld, fake(1), ld, fake(2), 2, eps, fake(3), ld,
                               fake(4), ld, at<float>(5), nullptr), "norm fwd");
            expect(rmsnorm_fwd(fake(0), dt, n, h, ld, nullptr, kMin, nullptr, dt, eps, fake(0), ld,
                               nullptr, kMax, nullptr, nullptr), "norm fwd, in place");
            expect(rmsnorm_fp8_fwd(fake(0), dt, n, h, ld, fake(1), ld, fake(2), 2, eps,
                                   at<uint8_t>(3), ld, fake(6), dt - 1, ld, fake(4), ld,
                                   at<float>(5), nullptr), "norm 8-bit fwd");
            expect(rmsnorm_bwd(fake(0), dt, ld, fake(1), ld, at<float>(2), fake(3), 2, fake(4), ld,
                               n, h, eps < 0, fake(5), ld, fake(6), 2, fake(7), big, nullptr),
                   "norm bwd");
            expect(rmsnorm_bwd(fake(0), dt, ld, fake(1), ld, at<float>(2), nullptr, dt, nullptr,
                               kMax, n, h, 0, nullptr, kMin, nullptr, dt, nullptr, 0, nullptr),
                   "norm bwd, nothing but checks");
            expect(fp8_quantize(fake(0), dt, n, h, ld, eps < 0 ? 128 : 1, at<uint8_t>(1), ld,
                                fake(2), dt - 1, ld, nullptr), "quantize");
          }
      for (int64_t k : kSizes) {
        expect(fp8_matmul_workspace_size(n, h, k, &bytes), "product ws", true);
        for (int64_t ld : kFew)
          for (int dt : {-1, 0, 2}) {
            expect(fp8_matmul(at<uint8_t>(0), ld, fake(1), ld, at<uint8_t>(2), ld, fake(3), ld,
                              dt ? 0 : 1, at<float>(4), n, h, k, fake(5), dt, ld, fake(6), big,
                              nullptr), "product");
            expect(fp8_matmul(at<uint8_t>(0), k, fake(1), n, at<uint8_t>(2), k, fake(3), k, 0,
                              nullptr, n, h, k, fake(5), dt, h, nullptr, 0, nullptr),
                   "product, no workspace");
          }
      }
      for (int64_t beams : kFew)
        for (int64_t num : kFew) {
          expect(beam_step_workspace_size(n, beams, h, num, &bytes), "beam ws", true);
          for (int64_t ld : kFew)
            expect(beam_step(fake(0), int(ld % 3), n, beams, h, ld, at<float>(1), at<uint8_t>(2),
                             int32_t(num % 7) - 1, num, -100, at<float>(3), at<int32_t>(4),
                             at<int32_t>(5), at<uint8_t>(6), at<int32_t>(7), fake(8), big, nullptr),
                   "beam step");
          for (int64_t run : {int64_t(0), int64_t(1), int64_t(16), int64_t(1) << 50, kMax})
            for (int64_t stride : kSizes) {
              const lce_beam_state s[] = {
                  {fake(1), fake(2), stride, run, h, stride, run, h, num, run},
                  {fake(3), fake(4), run, stride, h, run, stride, h, num, run}};
              expect(beam_reorder(s, 2, at<int32_t>(0), n, beams, beams, nullptr), "reorder", true);
              const lce_beam_state t[] = {
                  {fake(1), fake(1), stride, run, h, stride, run, h, num, run}};
              expect(beam_reorder(t, 1, at<int32_t>(0), n, beams, num, nullptr), "reorder", true);
            }
        }
    }
  // NULL, misaligned, undersized
  expect(rmsnorm_workspace_size(2, 16, nullptr), "norm ws NULL");
  expect(fp8_matmul_workspace_size(2, 16, 16, nullptr), "product ws NULL");
  expect(beam_step_workspace_size(2, 2, 16, 2, nullptr), "beam ws NULL");
  expect(rmsnorm_fwd(arena + 1, 0, 2, 16, 16, nullptr, 0, nullptr, 0, 0.f, fake(3), 16, nullptr, 0,
                     nullptr, nullptr), "norm fwd misaligned");
  expect(fp8_matmul(at<uint8_t>(0), 128, fake(1), 70, at<uint8_t>(2), 128, fake(3), 1, 0, nullptr,
                    70, 4096, 128, fake(5), 0, 4096, nullptr, 0, nullptr), "product misses");
  expect(beam_reorder(nullptr, 3, at<int32_t>(0), 2, 2, 2, nullptr), "reorder NULL");
  std::vector<lce_beam_state> many(size_t(1) << 16);
  for (size_t i = 0; i < many.size(); ++i)
    many[i] = {arena, arena + 65536 + i, 1 << 20, 1, 0, 1 << 20, 1, 0, 1, i % 3 ? 0 : 1};
  expect(beam_reorder(many.data(), int64_t(many.size()), at<int32_t>(0), 1, 1, 1, nullptr),
         "reorder of many");
  std::printf("%ld calls, %d failures\n", calls, failures);
  return failures ? 1 : 0;
}
