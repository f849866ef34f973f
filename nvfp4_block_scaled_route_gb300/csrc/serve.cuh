// Shared by the operators around a serving step (plan.cu, verify.cu) and the C-ABI
// layer, and what they use of thread-block clusters.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace nvmoe {

// A pool's free pages: `free` of them from ring[first] on, around its end.
struct PoolView {
  int32_t* ring;
  int64_t size;
  const int32_t* state;      // {first, free} before the step
  int32_t* state_out;        // ... after it; may be the same
};

struct PlanArgs {
  PoolView pool;
  int batch, page_shift;
  int64_t max_pages, rows;
  const int32_t* before;     // [batch] lengths after the step before; may be kv_len
  const int32_t* cached;     // [batch] how many of those tokens stand; may be either
  const int32_t* new_tokens; // [batch]; negative: the request ends
  int32_t* kv_len;           // [batch]
  int32_t* q_start;          // [batch + 1]
  int32_t* page_table;       // [batch, max_pages]
  int32_t* positions;        // [rows] or null
  int64_t* slots;            // [rows] or null
  int* status;
};
cudaError_t launch_plan_pages(const PlanArgs& args, cudaStream_t stream);

struct VerifyArgs {
  const void* target;        // [rows, vocab]
  const void* draft;         // [rows, vocab] or null
  bool bf16;                 // else fp32
  int64_t target_stride, draft_stride;   // elements
  int64_t rows;
  int vocab, batch;
  const int32_t* tokens;     // [rows]
  const int32_t* q_start;    // [batch + 1]
  const int32_t* kv_len;     // [batch] or null
  const float* accept_u;     // [rows]
  const float* sample_u;     // [batch]
  int32_t* accepted;         // [batch]
  int32_t* next_token;       // [batch]
  int32_t* cached;           // [batch] or null
  int* status;
};
cudaError_t launch_draft_verify(const VerifyArgs& args, cudaStream_t stream);

// ---- clusters ----
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
// A barrier of the cluster in two parts: arrive orders nothing, wait does.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// To the same place of CTA `rank`'s shared memory.
__device__ __forceinline__ void st_cluster_f32x2(void* p, uint32_t rank, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};"
               ::"r"(map_shared_rank(smem_u32(p), rank)), "f"(x), "f"(y) : "memory");
}

}  // namespace nvmoe
