// paged.cuh - the paged key/value cache: what its kernels share.
#pragma once

#include "common.cuh"
#include "tp3d_paged.h"

namespace tp3d {

// the most tokens of one request, and rows of one call: sums of a position and
// a few tiles' rows stay in 32 bits
constexpr int64_t kPagedMaxTokens = INT32_MAX - 4096;

// One call of tp3d_paged_attn, as its kernels take it (element strides).
struct PagedAttn {
  tp3d_kv_cache c;
  int32_t page_log2;
  int32_t requests, group;  // group: query heads per key/value head
  int32_t few_rows;         // requests with up to this many rows per key/value head go to the kernel for few
  int64_t tokens;
  const int32_t *q_start, *kv_len, *table;
  int64_t width;  // block table columns
  float scale;
  const __nv_bfloat16* q;
  int64_t q_token, q_head;
  __nv_bfloat16* o;
  int64_t o_token, o_head;
  float* lse;  // or null
  int* err;
  int64_t stall_after;  // test hook: the many-rows kernel's CTAs load this many key and value tiles each (-1: all)
};

tp3d_status launch_paged_attn(tp3d_ctx* ctx, PagedAttn& A, int max_new, void* workspace, cudaStream_t s);
size_t paged_attn_workspace(const tp3d_ctx* ctx, int head_dim);

#if defined(__CUDACC__)

// Programmatic dependent launch.  The paged kernels follow one another in a
// server's step and are short, so each is launched while the one before it on
// the stream still runs, and begins by waiting for that one's end (its memory
// is then visible); it lets the next one come as soon as it has.  All of a
// kernel's CTAs have begun by then, so those of the next never hold up its own.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// What an earlier kernel of the stream may have written is read with ordinary
// loads, which stay behind grid_wait; a read-only one (__ldg) may be moved, and
// wants data that nothing writes while the kernel runs, which begins early.
template <class T>
__device__ __forceinline__ T ld_plain(const T* p) {
  return *p;
}
__device__ __forceinline__ void grid_begin() {
  grid_wait();
  grid_launch_dependents();
}

template <class... Params, class... Args>
tp3d_status launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                             const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...) == cudaSuccess ? TP3D_OK : TP3D_ECUDA;
}

// A request as the attention kernels see it: rows [q0, q0 + n) of Q, kv keys.
// Lengths that do not fit are clamped, so that whatever the buffers hold, no
// access leaves them; a request that was clamped raises TP3D_EPAGES.
struct PagedRequest {
  int64_t q0;
  int32_t n, kv;
};
__device__ __forceinline__ PagedRequest paged_request(const PagedAttn& A, int b) {
  const int32_t s0 = ld_plain(A.q_start + b), s1 = ld_plain(A.q_start + b + 1), len = ld_plain(A.kv_len + b);
  const int64_t width = A.width << A.page_log2, cap = width < kPagedMaxTokens ? width : kPagedMaxTokens;
  PagedRequest r;
  const int64_t q0 = s0 < 0 ? 0 : s0 > A.tokens ? A.tokens : s0;
  const int64_t q1 = s1 < q0 ? q0 : s1 > A.tokens ? A.tokens : s1;
  r.q0 = q0;
  r.n = (int32_t)(q1 - q0);
  r.kv = (int32_t)(len < 0 ? 0 : len > cap ? cap : len);
  if (q0 != s0 || q1 != s1 || r.kv != len) raise_error(A.err, TP3D_EPAGES);
  return r;
}

#endif

}  // namespace tp3d
