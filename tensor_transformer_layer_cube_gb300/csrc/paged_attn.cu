// paged_attn.cu - attention of new tokens over the paged key/value cache.
//
// Row (t, i) of request b (new token j = t - q_start_b, query head i) sees
// the keys k = 0 .. kv_b - n_b + j:
//   s_k = scale q . k_k,  m = max s_k,  l = sum exp(s_k - m),
//   O = sum exp(s_k - m) v_k / l,  lse = m + log l,
// in one pass over the keys with a running m, l and O.
#include <math.h>

#include "paged.cuh"

namespace tp3d {

namespace {

using bf16 = __nv_bfloat16;

constexpr int kRowWarps = 4;

// One CTA per (row, query head); its warps take every kRowWarps-th key, each
// with its own running maximum and sums, joined at the end.  Lane l holds
// columns l * D/32 .. of the row.
template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) paged_attn_row_kernel(const PagedAttn A, int max_new) {
  constexpr int E = D / 32;
  __shared__ float so[kRowWarps][D], sm[kRowWarps], sl[kRowWarps];
  __shared__ int s_req;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.y, h = i / A.group;
  const int64_t t = blockIdx.x;
  if (threadIdx.x == 0) s_req = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < A.requests; b += kRowWarps * 32) {
    const PagedRequest r = paged_request(A, b);
    if (t >= r.q0 && t < r.q0 + r.n) s_req = b;
  }
  __syncthreads();
  const int b = s_req;
  if (b < 0) return;
  const PagedRequest r = paged_request(A, b);
  if (max_new > 0 && r.n > max_new) {
    raise_error(A.err, TP3D_EPAGES);
    return;
  }
  const int64_t last = (int64_t)r.kv - r.n + (t - r.q0);
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(A.q[t * A.q_token + i * A.q_head + lane * E + e]) * A.scale;
    o[e] = 0.0f;
  }
  for (int64_t k = warp; k <= last; k += kRowWarps) {
    const int32_t page = __ldg(A.table + (int64_t)b * A.width + (k >> A.page_log2));
    const bool in = page >= 0 && page < A.c.pages;
    if (!in) raise_error(A.err, TP3D_EPAGES);
    const int64_t at = (int64_t)page * A.c.page_stride + (k & (A.c.page - 1)) * A.c.token_stride +
                       h * A.c.head_stride + lane * E;
    const bf16* kp = static_cast<const bf16*>(A.c.k) + at;
    const bf16* vp = static_cast<const bf16*>(A.c.v) + at;
    float s = 0.0f;
    for (int e = 0; e < E; ++e) s += in ? q[e] * __bfloat162float(kp[e]) : 0.0f;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.0f : mn;
    const float f = expf(m - base), p = expf(s - base);
    l = l * f + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + (in ? p * __bfloat162float(vp[e]) : 0.0f);
    m = mn;
  }
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float mm = -INFINITY, ll = 0.0f;
  for (int w = 0; w < kRowWarps; ++w) mm = fmaxf(mm, sm[w]);
  const float base = mm == -INFINITY ? 0.0f : mm;
  for (int w = 0; w < kRowWarps; ++w) ll += sl[w] * expf(sm[w] - base);
  for (int c = threadIdx.x; c < D; c += kRowWarps * 32) {
    float x = 0.0f;
    for (int w = 0; w < kRowWarps; ++w) x += so[w][c] * expf(sm[w] - base);
    A.o[t * A.o_token + i * A.o_head + c] = __float2bfloat16(ll == 0.0f ? 0.0f : x / ll);
  }
  if (threadIdx.x == 0 && A.lse) A.lse[t * (int64_t)gridDim.y + i] = ll == 0.0f ? -INFINITY : base + logf(ll);
}

}  // namespace

size_t paged_attn_workspace(const tp3d_ctx*, int) { return 256; }

tp3d_status launch_paged_attn(tp3d_ctx*, const PagedAttn& A, int max_new, void*, cudaStream_t s) {
  const int heads = A.group * A.c.kv_heads;
  if (heads > 65535) return TP3D_EUNSUPPORTED;
  const dim3 grid((unsigned)A.tokens, (unsigned)heads);
  if (A.c.head_dim == 128)
    paged_attn_row_kernel<128><<<grid, kRowWarps * 32, 0, s>>>(A, max_new);
  else
    paged_attn_row_kernel<64><<<grid, kRowWarps * 32, 0, s>>>(A, max_new);
  return cudaGetLastError() == cudaSuccess ? TP3D_OK : TP3D_ECUDA;
}

}  // namespace tp3d
