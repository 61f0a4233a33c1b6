// PerIndex (csrc/per_device.h) on the host: values are made once for each index,
// by whichever thread comes first, and failures are not kept.
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

#define CHECK(x)                                     \
  do {                                               \
    if (!(x)) {                                      \
      std::printf("line %d: %s\n", __LINE__, #x);    \
      return 1;                                      \
    }                                                \
  } while (0)

int main() {
  static dg::PerIndex<int> slots;
  std::atomic<int> made[4] = {};
  std::atomic<int> wrong{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 16; ++t)
    threads.emplace_back([&, t] {
      for (int r = 0; r < 1000; ++r) {
        const int dev = (t + r) & 3;
        int v = -1;
        const cudaError_t e = slots.get(dev, &v, [&](int *out) {
          ++made[dev];
          *out = 100 + dev;
          return cudaSuccess;
        });
        if (e != cudaSuccess || v != 100 + dev) ++wrong;
      }
    });
  for (auto &t : threads) t.join();
  CHECK(wrong == 0);
  for (int dev = 0; dev < 4; ++dev) CHECK(made[dev] == 1);

  int v = -1, calls = 0;
  auto fails = [&](int *) { ++calls; return cudaErrorInvalidValue; };
  auto works = [&](int *out) { ++calls; *out = 7; return cudaSuccess; };
  CHECK(slots.get(9, &v, fails) == cudaErrorInvalidValue && v == -1);
  CHECK(slots.get(9, &v, works) == cudaSuccess && v == 7 && calls == 2);
  CHECK(slots.get(9, &v, fails) == cudaSuccess && v == 7 && calls == 2);
  for (int i : {-1, dg::kMaxDevices}) {   // outside the table: made at each call
    calls = 0;
    CHECK(slots.get(i, &v, works) == cudaSuccess && slots.get(i, &v, works) == cudaSuccess && calls == 2);
  }
  std::printf("ok\n");
  return 0;
}
