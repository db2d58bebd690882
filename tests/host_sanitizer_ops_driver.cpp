// Host-side exerciser of the embedding, layer norm and vocabulary-piece entry points, built with
// AddressSanitizer and UndefinedBehaviorSanitizer (tests/test_host_sanitizers_ops.py). As
// host_sanitizer_driver.cpp: extreme and inconsistent sizes, NULL and misaligned fake pointers,
// where no GPU is visible, so that a call which passes validation stops at the device check.
// Every call must return a documented code other than LCE_OK (size queries: a documented code).
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

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
const int64_t kSizes[] = {kMin, -1, 0, 1, 8, 1000, int64_t(1) << 20, (int64_t(1) << 23) + 1,
                          (int64_t(1) << 31) - 1, int64_t(1) << 31, int64_t(1) << 62, kMax};
const int64_t kFew[] = {-1, 1, 8, 4096, int64_t(1) << 20, (int64_t(1) << 31) - 1, kMax};

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
  for (int64_t n : kSizes) {
    expect(flce_piece_loss_workspace_size(n, &bytes), "piece loss ws", true);
    for (int64_t v : kSizes)
      expect(flce_piece_loss(at<float>(0), at<int32_t>(1), n, v, -100, -1, at<float>(2),
                             at<float>(3), at<float>(4), at<int32_t>(5), fake(6), big, nullptr),
             "piece loss");
    for (int64_t h : kSizes) {
      expect(layernorm_workspace_size(n, h, &bytes), "norm ws", true);
      for (int64_t ld : kSizes)
        for (int dt : {-1, 0, 1, 2, 3}) {
          expect(layernorm_fwd(fake(0), dt, n, h, ld, fake(1), fake(2), 2, 1e-5f, fake(3), ld,
                               at<float>(4), at<float>(5), nullptr), "norm fwd");
          expect(layernorm_bwd(fake(0), dt, ld, fake(1), ld, at<float>(2), at<float>(3), fake(4), 2,
                               n, h, 0, fake(5), ld, fake(6), fake(7), 2, fake(8), big, nullptr),
                 "norm bwd");
          expect(layernorm_bwd(fake(0), dt, ld, fake(1), ld, at<float>(2), at<float>(3), nullptr,
                               dt, n, h, 1, nullptr, kMax, nullptr, nullptr, dt, nullptr, 0,
                               nullptr), "norm bwd, nothing but checks");
        }
    }
    for (int64_t h : kSizes)
      for (int64_t v : kSizes) {
        expect(embed_workspace_size(n, h, v, &bytes), "embed ws", true);
        expect(flce_piece_fwd_workspace_size(n, h, v, &bytes), "piece fwd ws", true);
        expect(flce_piece_bwd_workspace_size(n, h, v, &bytes), "piece bwd ws", true);
        for (int64_t ld : kFew)
          for (int dt : {0, 2, 7}) {
            expect(embed_fwd(fake(0), dt, v, h, ld, at<int32_t>(1), n, -100, 1.f, fake(2), ld,
                             at<int32_t>(3), nullptr), "embed fwd");
            expect(embed_bwd(fake(0), dt, ld, at<int32_t>(1), n, h, v, -100, 1.f, 1, fake(2), 2, ld,
                             at<int32_t>(3), fake(4), big, nullptr), "embed bwd");
          }
        for (int64_t start : {kMin, int64_t(-1), int64_t(0), int64_t(1), kMax})
          for (int64_t vocab : {v, int64_t(1) << 31, kMax}) {
            expect(flce_piece_fwd(at<uint16_t>(0), at<uint16_t>(1), at<float>(2), at<int32_t>(3),
                                  n, h, v, start, vocab, -100, 1, at<float>(4), fake(5), big,
                                  nullptr), "piece fwd");
            expect(flce_piece_bwd(at<uint16_t>(0), at<uint16_t>(1), at<float>(2), at<int32_t>(3),
                                  at<float>(4), n, h, v, start, vocab, -100, -1, 7, at<float>(5),
                                  at<float>(6), at<float>(7), at<uint16_t>(8), fake(9), 2,
                                  at<float>(10), fake(11), big, nullptr), "piece bwd");
          }
      }
  }
  // NULL, misaligned, undersized
  expect(embed_fwd(nullptr, 0, 4, 8, 8, at<int32_t>(1), 2, -100, 1.f, fake(2), 8, nullptr, nullptr),
         "embed fwd NULL");
  expect(embed_bwd(fake(0), 0, 8, at<int32_t>(1), 2, 8, 4, -100, 1.f, 0, fake(2), 0, 8, nullptr,
                   fake(4), 1, nullptr), "embed bwd small workspace");
  expect(layernorm_fwd(arena + 1, 0, 2, 8, 8, nullptr, nullptr, 0, 0.f, fake(3), 8, nullptr, nullptr,
                       nullptr), "norm fwd misaligned");
  expect(flce_piece_bwd(at<uint16_t>(0), at<uint16_t>(1), nullptr, at<int32_t>(3), at<float>(4), 2,
                        8, 4, 0, 4, -100, -1, 2, nullptr, nullptr, nullptr, at<uint16_t>(8), nullptr,
                        0, nullptr, fake(11), big, nullptr), "piece bwd without hidden_acc");
  expect(embed_workspace_size(2, 8, 4, nullptr), "embed ws NULL");
  std::printf("%ld calls, %d failures\n", calls, failures);
  return failures ? 1 : 0;
}
