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
  int32_t window, sinks;  // keys that a row sees up to its own, and first ones that it sees besides (window 0: all)
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

constexpr int kPagedThreads = 256;  // of the kernels that are not attention

inline int page_log2(int page) {
  if (page < 16 || page > 4096 || (page & (page - 1))) return -1;
  int l = 4;
  while ((1 << l) < page) ++l;
  return l;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline tp3d_status check_cache(const tp3d_kv_cache* c) {
  if (!c || !c->k || !c->v || c->kv_heads < 1 || c->pages < 1) return TP3D_EINVAL;
  if (c->dtype != TP3D_BF16) return TP3D_EDTYPE;
  if ((c->head_dim != 64 && c->head_dim != 128) || page_log2(c->page) < 0 || c->pages > INT32_MAX)
    return TP3D_EUNSUPPORTED;
  if (c->page_stride < 1 || c->token_stride < 1 || c->head_stride < 1) return TP3D_EINVAL;
  if ((c->page_stride | c->token_stride | c->head_stride) >> 39) return TP3D_EUNSUPPORTED;  // a tensor map's strides
  if (!aligned16(c->k) || !aligned16(c->v) || (c->page_stride | c->token_stride | c->head_stride) % 8)
    return TP3D_EALIGN;
  return TP3D_OK;
}

// bytes from a strided (page, token, head) array's first element to its last;
// strides are the caller's and may be anything, so the sum is kept from
// wrapping (an array that long overlaps everything above it)
inline size_t extent(int64_t pages, int64_t ps, int64_t tokens, int64_t ts, int64_t heads, int64_t hs, int64_t d,
                     int elem_bytes = 2) {
  const unsigned __int128 n = ((unsigned __int128)(pages - 1) * (uint64_t)ps +
                               (unsigned __int128)(tokens - 1) * (uint64_t)ts +
                               (unsigned __int128)(heads - 1) * (uint64_t)hs + (uint64_t)d) *
                              (unsigned)elem_bytes;
  return n > (unsigned __int128)1 << 62 ? (size_t)1 << 62 : (size_t)n;
}
inline size_t cache_bytes(const tp3d_kv_cache& c) {
  return extent(c.pages, c.page_stride, c.page, c.token_stride, c.kv_heads, c.head_stride, c.head_dim);
}

struct Range {
  const void* p;
  size_t n;
};
// any output overlapping an input or another output
template <int NO, int NI>
bool clash(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
}

inline unsigned blocks(const tp3d_ctx* ctx, int64_t threads, int per_sm) {
  const int64_t n = (threads + kPagedThreads - 1) / kPagedThreads, most = (int64_t)ctx->num_sms * per_sm;
  return (unsigned)(n < 1 ? 1 : n < most ? n : most);
}

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

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void st_shared4(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// One thread's arrival for its CTA, whose writes before the last barrier come
// with it, at a count of `of` CTAs: whether it is the last (which sees all the
// others' writes, and lets the CTA see them by its next barrier).  The count
// returns to zero.
__device__ __forceinline__ bool arrive_last(unsigned* count, unsigned of) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(count), "r"(of - 1) : "memory");
  return old == of - 1;
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

__device__ __forceinline__ int32_t pages_of(int64_t n, int page_log2) {
  return (int32_t)((n + (1 << page_log2) - 1) >> page_log2);
}

// the last index i in [0, n) with a[i] <= x (a non-decreasing, a[0] <= x)
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
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
