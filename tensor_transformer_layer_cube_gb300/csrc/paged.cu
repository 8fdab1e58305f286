// paged.cu - the paged key/value cache: block tables and slot maps from
// request lengths, the cache write, and the entry points of
// include/tp3d_paged.h.
#include <math.h>

#include "paged.cuh"

namespace tp3d {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ plan
// With c_b cached and f_b new tokens, old_b = ceil(c_b / page) and
// need_b = ceil((c_b + f_b) / page) - old_b, everything a step needs follows
// from the exclusive sums of f and of need over the requests: new page i of
// the step (request by request) is free[count - 1 - i], and a new token
// finds its request by a search in the sums of f.  So one launch does it all:
// every CTA forms both sums in shared memory (8 bytes per request read from
// L2, 8 kept), then takes its share of the new table entries and of the
// tokens.  No CTA reads what another writes: a token's page is an old table
// entry or, for a new page, the free list entry again.
//
// It moves 16 bytes per request and 12 per token, so launch latency and the
// two dependent reads (lengths, then free list or table) bound it: 256 requests
// of one token 3.4 us on the GPU, 64 prompts (48467 tokens) 3.8 us; the
// host takes 5.9 us a call.
constexpr int kScanItems = 4;
constexpr int kScanChunk = kThreads * kScanItems;
constexpr int kPlanMaxRequests = 16384;
constexpr int kPlanReady = 4;  // of tp3d_ctx::paged_ready

struct PlanArgs {
  int page_log2, requests;
  int64_t tokens;
  const int32_t *cached, *fresh, *free_pages;
  int64_t free_cap;
  const int32_t* free_count;
  int32_t* table;
  int64_t width;
  int32_t *q_start, *kv_len;
  int64_t* slots;
  int32_t* positions;
  int32_t* free_left;
  int* err;
};

struct Lengths {
  int32_t cached, fresh;
  bool bad;
};
// The lengths of request b; bad ones take no new tokens.
__device__ __forceinline__ Lengths plan_lengths(const PlanArgs& P, int b) {
  Lengths l{ld_plain(P.cached + b), ld_plain(P.fresh + b), false};
  const int64_t cap = P.width << P.page_log2, kv = (int64_t)l.cached + l.fresh;
  if (l.cached < 0 || l.fresh < 0 || kv > cap || kv > kPagedMaxTokens) {
    l.bad = true;
    l.fresh = 0;
    l.cached = l.cached < 0 ? 0 : l.cached > cap ? (int32_t)(cap < kPagedMaxTokens ? cap : kPagedMaxTokens) : l.cached;
  }
  return l;
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

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const PlanArgs P) {
  extern __shared__ int32_t plan_smem[];
  int32_t* sf = plan_smem;                    // exclusive sums of fresh, requests + 1
  int32_t* sp = plan_smem + P.requests + 1;   // exclusive sums of the new pages, requests + 1
  __shared__ long long warp_f[kThreads / 32], warp_p[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool first = blockIdx.x == 0;
  grid_begin();
  const int64_t count0 = ld_plain(P.free_count);
  const int64_t count = count0 < 0 ? 0 : count0 > P.free_cap ? P.free_cap : count0;

  bool bad = count != count0;
  long long carry_f = 0, carry_p = 0;  // 64-bit: the sums of bad input may pass 32 bits
  for (int base = 0; base < P.requests; base += kScanChunk) {
    const int b0 = base + (int)threadIdx.x * kScanItems;
    int32_t f[kScanItems], p[kScanItems];
    long long tf = 0, tp = 0;
#pragma unroll
    for (int i = 0; i < kScanItems; ++i) {
      f[i] = p[i] = 0;
      if (b0 + i < P.requests) {
        const Lengths l = plan_lengths(P, b0 + i);
        bad |= l.bad;
        f[i] = l.fresh;
        p[i] = pages_of((int64_t)l.cached + l.fresh, P.page_log2) - pages_of(l.cached, P.page_log2);
        if (first) P.kv_len[b0 + i] = l.cached + l.fresh;
      }
      tf += f[i];
      tp += p[i];
    }
    long long xf = tf, xp = tp;  // inclusive sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long yf = __shfl_up_sync(0xffffffffu, xf, o), yp = __shfl_up_sync(0xffffffffu, xp, o);
      if (lane >= o) {
        xf += yf;
        xp += yp;
      }
    }
    if (lane == 31) {
      warp_f[warp] = xf;
      warp_p[warp] = xp;
    }
    __syncthreads();
    long long bf = carry_f + xf - tf, bp = carry_p + xp - tp;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        bf += warp_f[w];
        bp += warp_p[w];
      }
      carry_f += warp_f[w];
      carry_p += warp_p[w];
    }
#pragma unroll
    for (int i = 0; i < kScanItems; ++i) {
      if (b0 + i < P.requests) {
        sf[b0 + i] = (int32_t)(bf < INT32_MAX ? bf : INT32_MAX);
        sp[b0 + i] = (int32_t)(bp < INT32_MAX ? bp : INT32_MAX);
        if (first) P.q_start[b0 + i] = sf[b0 + i];
      }
      bf += f[i];
      bp += p[i];
    }
    __syncthreads();
  }
  const int32_t total_f = (int32_t)(carry_f < INT32_MAX ? carry_f : INT32_MAX);
  const int32_t total_p = (int32_t)(carry_p < INT32_MAX ? carry_p : INT32_MAX);
  bad |= carry_f > P.tokens || carry_f > INT32_MAX || carry_p > count;
  if (first) {
    if (bad) raise_error(P.err, TP3D_EPAGES);
    if (threadIdx.x == 0) {
      P.q_start[P.requests] = total_f;
      *P.free_left = (int32_t)(carry_p < count ? count - carry_p : 0);
    }
  }

  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = tid; i < total_p; i += step) {
    const int b = last_at_most(sp, P.requests, (int32_t)i);
    const Lengths l = plan_lengths(P, b);
    const int64_t col = pages_of(l.cached, P.page_log2) + (i - sp[b]);
    P.table[(int64_t)b * P.width + col] = i < count ? ld_plain(P.free_pages + (count - 1 - i)) : -1;
  }
  for (int64_t t = tid; t < P.tokens; t += step) {
    int64_t slot = -1;
    int32_t pos = 0;
    if (t < total_f) {
      const int b = last_at_most(sf, P.requests, (int32_t)t);
      const Lengths l = plan_lengths(P, b);
      pos = l.cached + (int32_t)(t - sf[b]);
      const int32_t col = pos >> P.page_log2, old = pages_of(l.cached, P.page_log2);
      const int64_t i = (int64_t)sp[b] + (col - old);  // the step's new page number, if new
      const int32_t page = col < old ? P.table[(int64_t)b * P.width + col]
                                     : i < count ? ld_plain(P.free_pages + (count - 1 - i)) : -1;
      if (page >= 0) slot = ((int64_t)page << P.page_log2) + (pos & ((1 << P.page_log2) - 1));
    }
    P.slots[t] = slot;
    P.positions[t] = pos;
  }
}

// ------------------------------------------------------------------ store
// A copy of 16-byte vectors, K and V in one launch: consecutive threads take
// the consecutive vectors of a (token, head) row, and each has kStoreVecs
// vectors of K and of V in flight.  HBM-bound for many tokens (16385 of 8 heads
// of 128, 134 MB: 22.8 us, 0.88 of the copy rate; with one vector in flight
// 24.5), launch latency for few (64 tokens: 1.5 us on the GPU, 5.1 us a call).
struct StoreArgs {
  tp3d_kv_cache c;
  int page_log2, vec_log2;  // 16-byte vectors of a row: 1 << vec_log2
  int64_t tokens, token_stride, head_stride;
  const __nv_bfloat16 *k, *v;
  const int64_t* slots;
  int* err;
};

constexpr int kStoreVecs = 4;  // of K and of V each, in flight per thread

__global__ void __launch_bounds__(kThreads) paged_store_kernel(const StoreArgs S) {
  grid_begin();
  const int64_t rows = S.tokens * S.c.kv_heads, total = rows << S.vec_log2;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += kStoreVecs * step) {
    uint4 k[kStoreVecs], v[kStoreVecs];
    int64_t to[kStoreVecs];
#pragma unroll
    for (int q = 0; q < kStoreVecs; ++q) {
      const int64_t i = i0 + q * step;
      to[q] = -1;
      if (i >= total) continue;
      const int vec = (int)(i & ((1 << S.vec_log2) - 1)) * 8;
      const int64_t row = i >> S.vec_log2;
      // 32-bit division where it fits: a 64-bit one costs as much as the copy
      const int64_t t = row >> 32 ? row / S.c.kv_heads : (int64_t)((uint32_t)row / (uint32_t)S.c.kv_heads);
      const int h = (int)(row - t * S.c.kv_heads);
      const int64_t slot = ld_plain(S.slots + t), page = slot >> S.page_log2;
      if (slot < 0) continue;
      if (page >= S.c.pages) {
        raise_error(S.err, TP3D_EPAGES);
        continue;
      }
      to[q] = page * S.c.page_stride + (slot & ((1 << S.page_log2) - 1)) * S.c.token_stride + h * S.c.head_stride + vec;
      const int64_t from = t * S.token_stride + h * S.head_stride + vec;
      k[q] = ld_plain(reinterpret_cast<const uint4*>(S.k + from));
      v[q] = ld_plain(reinterpret_cast<const uint4*>(S.v + from));
    }
#pragma unroll
    for (int q = 0; q < kStoreVecs; ++q) {
      if (to[q] < 0) continue;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(S.c.k) + to[q]) = k[q];
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(S.c.v) + to[q]) = v[q];
    }
  }
}

int page_log2(int page) {
  if (page < 16 || page > 4096 || (page & (page - 1))) return -1;
  int l = 4;
  while ((1 << l) < page) ++l;
  return l;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

tp3d_status check_cache(const tp3d_kv_cache* c) {
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
size_t extent(int64_t pages, int64_t ps, int64_t tokens, int64_t ts, int64_t heads, int64_t hs, int64_t d) {
  const unsigned __int128 n = ((unsigned __int128)(pages - 1) * (uint64_t)ps +
                               (unsigned __int128)(tokens - 1) * (uint64_t)ts +
                               (unsigned __int128)(heads - 1) * (uint64_t)hs + (uint64_t)d) * 2;
  return n > (unsigned __int128)1 << 62 ? (size_t)1 << 62 : (size_t)n;
}
size_t cache_bytes(const tp3d_kv_cache& c) {
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

unsigned blocks(const tp3d_ctx* ctx, int64_t threads, int per_sm) {
  const int64_t n = (threads + kThreads - 1) / kThreads, most = (int64_t)ctx->num_sms * per_sm;
  return (unsigned)(n < 1 ? 1 : n < most ? n : most);
}

}  // namespace

}  // namespace tp3d

using namespace tp3d;

extern "C" {

tp3d_status tp3d_paged_plan(tp3d_ctx* ctx, int page, int requests, int64_t tokens, const int32_t* cached,
                            const int32_t* fresh, const int32_t* free_pages, int64_t free_cap,
                            const int32_t* free_count, int32_t* block_table, int64_t table_width, int32_t* q_start,
                            int32_t* kv_len, int64_t* slots, int32_t* positions, int32_t* free_left, void* stream) {
  if (!ctx || !free_count || !q_start || !free_left) return TP3D_EINVAL;
  if (requests < 0 || tokens < 0 || free_cap < 0 || table_width < 0) return TP3D_EINVAL;
  if (requests > 0 && (!cached || !fresh || !block_table || !kv_len)) return TP3D_EINVAL;
  if ((tokens > 0 && (!slots || !positions)) || (free_cap > 0 && !free_pages)) return TP3D_EINVAL;
  const int pl = page_log2(page);
  if (pl < 0 || requests > kPlanMaxRequests || tokens > INT32_MAX || table_width > INT32_MAX ||
      free_cap > INT32_MAX)
    return TP3D_EUNSUPPORTED;
  const void* words[] = {cached, fresh, free_pages, free_count, block_table, q_start, kv_len, positions, free_left};
  for (const void* p : words)
    if (!aligned(p, 4)) return TP3D_EALIGN;
  if (!aligned(slots, 8)) return TP3D_EALIGN;
  const size_t rb = (size_t)requests * 4;
  const Range out[] = {{block_table, rb * (size_t)table_width}, {q_start, rb + 4}, {kv_len, rb},
                       {slots, (size_t)tokens * 8}, {positions, (size_t)tokens * 4}, {free_left, 4}};
  const Range in[] = {{cached, rb}, {fresh, rb}, {free_pages, (size_t)free_cap * 4}, {free_count, 4}};
  if (clash(out, in)) return TP3D_EOVERLAP;
  const PlanArgs P{pl, requests, tokens, cached, fresh, free_pages, free_cap, free_count, block_table, table_width,
                   q_start, kv_len, slots, positions, free_left, ctx->d_err};
  const size_t smem = ((size_t)requests + 1) * 8;
  // The limit is the function's, and so every context's and host thread's: set to the largest size once, never lowered.
  if (smem > 48 * 1024 && !(ctx->paged_ready & kPlanReady)) {
    TP3D_CUDA_TRY(cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (kPlanMaxRequests + 1) * 8));
    ctx->paged_ready |= kPlanReady;
  }
  return launch_dependent(paged_plan_kernel, blocks(ctx, tokens, 1), kThreads, smem, as_stream(stream), P);
}

tp3d_status tp3d_paged_store(tp3d_ctx* ctx, const tp3d_kv_cache* cache, int64_t tokens, const void* K, const void* V,
                             int64_t token_stride, int64_t head_stride, const int64_t* slots, void* stream) {
  if (!ctx || tokens < 0) return TP3D_EINVAL;
  TP3D_TRY(check_cache(cache));
  if (tokens == 0) return TP3D_OK;
  if (!K || !V || !slots || token_stride < 0 || head_stride < 0) return TP3D_EINVAL;
  if (!aligned16(K) || !aligned16(V) || (token_stride | head_stride) % 8 || !aligned(slots, 8)) return TP3D_EALIGN;
  const size_t cb = cache_bytes(*cache);
  const size_t nb = extent(1, 0, tokens, token_stride, cache->kv_heads, head_stride, cache->head_dim);
  const Range out[] = {{cache->k, cb}, {cache->v, cb}};
  const Range in[] = {{K, nb}, {V, nb}, {slots, (size_t)tokens * 8}};
  // the two pools may share one allocation (interleaved pages), so only inputs are checked against them
  for (const Range& o : out)
    for (const Range& i : in)
      if (overlaps(o.p, o.n, i.p, i.n)) return TP3D_EOVERLAP;
  const StoreArgs S{*cache, page_log2(cache->page), cache->head_dim == 128 ? 4 : 3, tokens, token_stride, head_stride,
                    static_cast<const __nv_bfloat16*>(K), static_cast<const __nv_bfloat16*>(V), slots, ctx->d_err};
  const int64_t vecs = tokens * cache->kv_heads * (cache->head_dim / 8);
  return launch_dependent(paged_store_kernel, blocks(ctx, vecs, 8), kThreads, 0, as_stream(stream), S);
}

size_t tp3d_paged_attn_workspace_bytes(tp3d_ctx* ctx, const tp3d_kv_cache* cache, int heads) {
  if (!ctx || check_cache(cache) != TP3D_OK || heads < 1 || heads % cache->kv_heads) return 0;
  return paged_attn_workspace(ctx, cache->head_dim);
}

tp3d_status tp3d_paged_attn(tp3d_ctx* ctx, const tp3d_kv_cache* cache, const tp3d_paged_batch* batch, int heads,
                            float scale, const void* Q, tp3d_row_strides q_strides, void* O,
                            tp3d_row_strides o_strides, float* lse, void* workspace, void* stream) {
  if (!ctx || !batch || heads < 1) return TP3D_EINVAL;
  TP3D_TRY(check_cache(cache));
  if (!(scale > 0.0f) || !isfinite(scale)) return TP3D_EINVAL;
  if (heads % cache->kv_heads) return TP3D_ESHAPE;
  if (heads / cache->kv_heads > 128) return TP3D_EUNSUPPORTED;
  if (batch->requests < 0 || batch->tokens < 0 || batch->table_width < 0) return TP3D_EINVAL;
  if (batch->tokens > kPagedMaxTokens || batch->table_width > INT32_MAX) return TP3D_EUNSUPPORTED;
  if (batch->requests == 0 || batch->tokens == 0) return TP3D_OK;
  if (!batch->q_start || !batch->kv_len || (batch->table_width > 0 && !batch->block_table)) return TP3D_EINVAL;
  if (!Q || !O || !workspace) return TP3D_EINVAL;
  if (q_strides.token_stride < 1 || q_strides.head_stride < 1 || o_strides.token_stride < 1 ||
      o_strides.head_stride < 1)
    return TP3D_EINVAL;
  if ((q_strides.token_stride | q_strides.head_stride) >> 39) return TP3D_EUNSUPPORTED;
  if (!aligned16(Q) || !aligned16(O) || !aligned(workspace, 256) || !aligned(lse, 4) ||
      !aligned(batch->q_start, 4) || !aligned(batch->kv_len, 4) || !aligned(batch->block_table, 4))
    return TP3D_EALIGN;
  if ((q_strides.token_stride | q_strides.head_stride | o_strides.token_stride | o_strides.head_stride) % 8)
    return TP3D_EALIGN;
  const int d = cache->head_dim;
  const size_t rb = (size_t)batch->requests * 4, cb = cache_bytes(*cache);
  const Range out[] = {{O, extent(1, 0, batch->tokens, o_strides.token_stride, heads, o_strides.head_stride, d)},
                       {lse, (size_t)batch->tokens * heads * 4},
                       {workspace, paged_attn_workspace(ctx, d)}};
  const Range in[] = {{Q, extent(1, 0, batch->tokens, q_strides.token_stride, heads, q_strides.head_stride, d)},
                      {cache->k, cb}, {cache->v, cb}, {batch->q_start, rb + 4}, {batch->kv_len, rb},
                      {batch->block_table, rb * (size_t)batch->table_width}};
  if (clash(out, in)) return TP3D_EOVERLAP;
  PagedAttn A{};
  A.c = *cache;
  A.page_log2 = page_log2(cache->page);
  A.requests = batch->requests;
  A.group = heads / cache->kv_heads;
  A.tokens = batch->tokens;
  A.q_start = batch->q_start;
  A.kv_len = batch->kv_len;
  A.table = batch->block_table;
  A.width = batch->table_width;
  A.scale = scale;
  A.q = static_cast<const __nv_bfloat16*>(Q);
  A.q_token = q_strides.token_stride;
  A.q_head = q_strides.head_stride;
  A.o = static_cast<__nv_bfloat16*>(O);
  A.o_token = o_strides.token_stride;
  A.o_head = o_strides.head_stride;
  A.lse = lse;
  A.err = ctx->d_err;
  A.stall_after = ctx->stall_after;
  return launch_paged_attn(ctx, A, batch->max_new, workspace, as_stream(stream));
}

}  // extern "C"
