// Host-side checks that the entry points of include/mha_paged.h share.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "../../include/mha_paged.h"
#include "host.cuh"

namespace mha {
namespace {

constexpr size_t kAlign = 256;
inline size_t round_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// One argument's memory: where, how much, the alignment it needs.
struct Buffer {
  const void *p;
  size_t n;
  size_t align;
};

// Whether every buffer with a size is there and aligned.
template <size_t N>
bool present(const Buffer (&bufs)[N]) {
  for (const Buffer &b : bufs)
    if (b.n > 0 && (b.p == nullptr || reinterpret_cast<uintptr_t>(b.p) % b.align != 0)) return false;
  return true;
}

// Whether an output shares memory with an input or another output; output i may
// be input in_place[i] itself (same address).
template <size_t N, size_t M>
bool clash(const Buffer (&outs)[N], const Buffer (&ins)[M], const int (&in_place)[N]) {
  for (size_t o = 0; o < N; ++o) {
    for (size_t i = 0; i < M; ++i) {
      if (static_cast<int>(i) == in_place[o] && outs[o].p == ins[i].p) continue;
      if (overlaps(outs[o].p, outs[o].n, ins[i].p, ins[i].n)) return true;
    }
    for (size_t o2 = o + 1; o2 < N; ++o2)
      if (overlaps(outs[o].p, outs[o].n, outs[o2].p, outs[o2].n)) return true;
  }
  return false;
}

// Whether a product of counts (>= 0) stays below 2^56: sizes in bytes then fit.
inline bool fits(std::initializer_list<long long> counts) {
  long long n = 1;
  for (const long long c : counts) {
    if (c != 0 && n > (1LL << 56) / c) return false;
    n *= c;
  }
  return true;
}

inline size_t elem_size(int dtype) { return dtype == MHA_DTYPE_F32 ? 4 : 2; }

// SMs of the current device; 0 on failure
inline int current_sms() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess ? sm_count(dev) : 0;
}

}  // namespace
}  // namespace mha
