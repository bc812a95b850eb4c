// Host-side services that the entry points of the library share (defined in
// mha_api.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mha {

// Number of SMs of a device (cached); 0 on failure.
int sm_count(int dev);

// Device address of the current device's status word; nullptr on failure.
int *status_ptr();

// Wait limit of the kernels' bounded waits (mha_debug_set_wait).
uint64_t wait_limit_ns();
int wait_stall();  // ... and its stall bits

// 4-D view (d, L, heads, B) of a contiguous bf16 tensor in either layout,
// 128-byte swizzle; box (64, box_rows, box_heads, 1)
bool make_map(CUtensorMap *map, const void *base, int d, int L, int heads, int B, int layout,
              int box_rows, int box_heads);

// Whether [a, a + na) and [b, b + nb) share a byte (null and empty ranges do not).
bool overlaps(const void *a, size_t na, const void *b, size_t nb);

}  // namespace mha
