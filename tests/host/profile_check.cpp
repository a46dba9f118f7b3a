// Host check of the timing facility's readers: flce_profile.cpp with stand-ins
// for the HIP event calls.  A caller's arrays are written up to their length
// and no further, whatever number of kernel kinds the library knows.
#include <cstdio>

#include "flce_internal.hpp"

static int events = 0;
extern "C" {
hipError_t hipEventCreate(hipEvent_t* e) { *e = reinterpret_cast<hipEvent_t>(static_cast<intptr_t>(++events)); return hipSuccess; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
hipError_t hipEventElapsedTime(float* ms, hipEvent_t, hipEvent_t) { *ms = 2.0f; return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
}

static int failed = 0;
#define CHECK(c) ((c) ? (void)0 : (void)(++failed, std::printf("line %d: %s\n", __LINE__, #c)))

int main() {
  constexpr int kRoom = 64;
  double ms[kRoom];
  int64_t count[kRoom];
  auto clear = [&] {
    for (int i = 0; i < kRoom; ++i) {
      ms[i] = -1.0;
      count[i] = -1;
    }
  };
  auto untouched_from = [&](int n) {
    for (int i = n; i < kRoom; ++i)
      if (ms[i] != -1.0 || count[i] != -1) return false;
    return true;
  };
  auto run = [] {
    for (int k = 0; k < FLCE_KERNEL_KINDS; ++k)
      for (int i = 0; i <= k; ++i) flce::ProfileScope ps(k, nullptr);
  };
  CHECK(flce_profile_enable(1) == FLCE_OK);
  run();
  clear();
  CHECK(flce_profile_read(nullptr, ms, count, 0) == FLCE_OK);
  CHECK(untouched_from(12));   // the kinds of a program built against the first header
  for (int k = 0; k < 12; ++k) CHECK(count[k] == k + 1 && ms[k] == 2.0 * (k + 1));
  for (int n : {0, 1, 12, int(FLCE_KERNEL_KINDS), kRoom - 1}) {
    clear();
    CHECK(flce_profile_read_n(nullptr, ms, count, n, 0) == FLCE_OK);
    CHECK(untouched_from(n));
    for (int k = 0; k < n; ++k) {
      const bool known = k < FLCE_KERNEL_KINDS;
      CHECK(count[k] == (known ? k + 1 : 0) && ms[k] == (known ? 2.0 * (k + 1) : 0.0));
    }
  }
  // a reset clears every kind, also through the shorter call
  CHECK(flce_profile_read(nullptr, ms, count, 1) == FLCE_OK);
  CHECK(flce_profile_read_n(nullptr, ms, count, FLCE_KERNEL_KINDS, 0) == FLCE_OK);
  for (int k = 0; k < FLCE_KERNEL_KINDS; ++k) CHECK(count[k] == 0 && ms[k] == 0.0);
  CHECK(flce_profile_read_n(nullptr, ms, count, -1, 0) == FLCE_EINVAL);
  CHECK(flce_profile_read_n(nullptr, nullptr, count, 1, 0) == FLCE_EINVAL);
  CHECK(flce_profile_read_n(nullptr, ms, nullptr, 1, 0) == FLCE_EINVAL);
  CHECK(flce_profile_read(nullptr, nullptr, nullptr, 0) == FLCE_EINVAL);
  std::printf("%d failed checks\n", failed);
  return failed != 0;
}
