// What the forward-pass kernels found wrong in their lists.  They run on streams of the caller's
// choice, so one may report while hc_pool_sync takes the reports of others: there is a 64-bit word
// per kind, the smallest position reported since it was last taken, kNothing when there is none.
// A report is one atomic minimum and a taking one atomic exchange of the same word, so a report is
// either in what is taken or stays for the next time, and keeps its position.
// `Atomic`: minimum and exchange of such a word, on the device its atomics.
#pragma once

#include <stdint.h>

namespace hc {

enum Wrong { kWrongIndex = 0, kWrongLengths = 1, kWrongKinds = 2 };  // out of range; a sequence's lengths
typedef unsigned long long WrongWord;
constexpr WrongWord kNothing = ~0ull;

#if defined(__HIP__)
#define HC_DEVICE __device__ __forceinline__
struct DeviceAtomic {
  static __device__ __forceinline__ void minimum(WrongWord* word, WrongWord x) { atomicMin(word, x); }
  static __device__ __forceinline__ WrongWord exchange(WrongWord* word, WrongWord x) { return atomicExch(word, x); }
};
#else
#define HC_DEVICE inline
#endif

template <class Atomic>
HC_DEVICE void report_wrong(WrongWord* words, Wrong kind, int64_t position) {
  Atomic::minimum(words + kind, (WrongWord)position);
}

template <class Atomic>
HC_DEVICE void take_wrong(WrongWord* words, WrongWord* taken) {
  for (int k = 0; k < kWrongKinds; k++) taken[k] = Atomic::exchange(words + k, kNothing);
}

#undef HC_DEVICE

// What hc_pool_sync takes: error bits and smallest position of the transfers, the forward pass's words.
struct TakenReports {
  WrongWord bits, position, words[kWrongKinds];
};

// The bits of HC_ERR_DEVICE's code that reports stand for, and their smallest position.
inline int wrong_code(const WrongWord* words, WrongWord* position) {
  static const int bits[kWrongKinds] = {1, 4};
  int code = 0;
  for (int k = 0; k < kWrongKinds; k++) {
    if (words[k] == kNothing) continue;
    code |= bits[k];
    if (words[k] < *position) *position = words[k];
  }
  return code;
}

}  // namespace hc
