// The entry points of include/mha_paged.h around recorded launches: what paged_api.cu hands to
// its kernels, without a GPU.  The device that it asks for is number 0, with 152 SMs.
#include <cuda_runtime.h>

static cudaError_t device_zero(int *dev) {
  *dev = 0;
  return cudaSuccess;
}
#define cudaGetDevice device_zero
#include "paged_api.cu"
#undef cudaGetDevice

namespace {
RopeArgs rope;
PagedProblem problem;
int kernel, launched, merged;  // 1 fp32, 2 few, 3 many; its CTAs; launches of the merge
}  // namespace

namespace mha {
int sm_count(int) { return 152; }
int *status_ptr() {
  static int word;
  return &word;
}
uint64_t wait_limit_ns() { return 1; }
int wait_stall() { return 0; }
bool make_map(CUtensorMap *, const void *, int, int, int, int, int, int, int) { return true; }
bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && na > 0 && nb > 0 && x < y + nb && y < x + na;
}
cudaError_t launch_rope_fwd(const RopeArgs &a, int, int, bool, int, cudaStream_t) {
  rope = a;
  return cudaSuccess;
}
cudaError_t launch_rope_bwd(const RopeArgs &a, int, int, int, cudaStream_t) {
  rope = a;
  return cudaSuccess;
}
static cudaError_t attention(const PagedProblem &p, int which, int grid) {
  problem = p;
  kernel = which;
  launched = grid;
  merged = 0;
  return cudaSuccess;
}
cudaError_t launch_paged_few(const CUtensorMap &, const CUtensorMap &, const CUtensorMap &,
                             const PagedProblem &p, int, int &grid, int, cudaStream_t) {
  return attention(p, 2, grid);
}
cudaError_t launch_paged_many(const CUtensorMap &, const CUtensorMap &, const CUtensorMap &,
                              const PagedProblem &p, int, int grid, cudaStream_t) {
  return attention(p, 3, grid);
}
cudaError_t launch_paged_simt(const PagedProblem &p, int, int grid, cudaStream_t) {
  return attention(p, 1, grid);
}
cudaError_t launch_paged_merge(const PagedProblem &, int, int, bool, int, int, cudaStream_t) {
  ++merged;
  return cudaSuccess;
}
}  // namespace mha

extern "C" {
// of the last row operator
const void *rope_q_weight() { return rope.q_weight; }
const void *rope_k_weight() { return rope.k_weight; }
// of the last attention
int attention_kernel() { return kernel; }
int attention_rows() { return problem.rows; }
int attention_tokens() { return problem.tb; }
int attention_ctas() { return launched; }
int attention_merged() { return merged; }
// bytes behind the workspace's begin that its slots end at
long long attention_slots_end(int d) {
  return reinterpret_cast<const char *>(paged_slot_ptr(problem, d, launched, 0)) -
         reinterpret_cast<const char *>(problem.meta);
}
}
