// rope.cu - the norm of query and key heads with the rotation by position:
// forward, backward, and the form that writes keys and values to the paged
// cache (include/tp3d_rope.h, tp3d_paged_rope_store of include/tp3d_paged.h).
//
// Row x of one head at position p: n = x s w with s = 1 / sqrt(mean x^2 + eps),
// y = R(p) n.  R turns pairs of columns by p f_j; with the frequency as a 64-bit
// fraction F of a turn, the angle is p F mod 2^64: an integer product that
// drops whole turns by itself, of which the upper 32 bits are as many as fp32
// can use.
//
// Every element is read once and written once, so HBM bounds many tokens and
// latency few.  A row's columns lie on LANES neighbouring lanes, eight each (16
// bytes of bf16), so the sums of a row and the partner columns of its pairs
// are shuffles within a warp.  A warp takes one token and goes over its heads,
// 32 / LANES at a time: the angles of its columns are computed once for all of
// them (eight sines and cosines a lane, some 200 instructions, against 100 for each
// head).  Where tokens are few, several warps share a token's heads.
#include <math.h>

#include "paged.cuh"

namespace tp3d {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeFlight = 4;  // rows that a lane has in flight
constexpr int kBackThreads = 512;

struct RowsIn {
  const void* p;
  int64_t token, head;
};
struct RowsOut {
  void* p;
  int64_t token, head;
};

struct RopeArgs {
  int32_t tokens, heads, kv_heads, dim, rot, norm, split;  // split: warps that share a token's heads
  float eps, magnitude;
  const uint64_t* turns;
  const void *qw, *kw;
  const int32_t* positions;
  RowsIn q, k, v;  // v: of the store form
  RowsOut qo, ko;
  // store form
  tp3d_kv_cache c;
  int page_log2;
  const int64_t* slots;
  int* err;
  // backward: q, k are the forward's inputs, dq, dk its results' gradients
  RowsIn dq, dk;
  void *dqw, *dkw;
  float* parts;
  unsigned* arrivals;
};

// eight columns of a row as they lie in memory
template <class T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = ld_plain(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void load(const float* p) {
    a = ld_plain(reinterpret_cast<const float4*>(p));
    b = ld_plain(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// A lane's eight columns from column c: their cosines and sines at one position.
// Halves: columns c + e turn against those rotary_dim / 2 away, eight angles;
// interleaved: pairs inside the eight, four.
template <bool INTER>
struct Turn {
  float cs[INTER ? 4 : 8], sn[INTER ? 4 : 8];
  bool turns;   // these columns are turned
  int partner;  // the lane of the other columns (halves)
  __device__ __forceinline__ void place(int rot, int c, int lane) {
    turns = c < rot;
    partner = !turns ? lane : c < rot / 2 ? lane + rot / 16 : lane - rot / 16;
  }
  // sign -1: the transposed rotation
  __device__ __forceinline__ void at(const RopeArgs& A, int pos, int c, float sign) {
    if (!turns) return;
    const int half = A.rot / 2, j0 = INTER ? c / 2 : c < half ? c : c - half;
    const float up = INTER || c >= half ? sign : -sign;  // the first column of a pair gets minus the sine
#pragma unroll
    for (int e = 0; e < (INTER ? 4 : 8); ++e) {
      const uint64_t turn = (uint64_t)(int64_t)pos * ld_plain(A.turns + j0 + e);
      // half turns in [-1, 1]
      sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 0x1p-31f, &sn[e], &cs[e]);
      cs[e] *= A.magnitude;
      sn[e] *= up * A.magnitude;
    }
  }
  // x turned; all lanes of the warp take part
  __device__ __forceinline__ void apply(float (&x)[8]) const {
    if (INTER) {
      if (!turns) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = fmaf(a, cs[i & 3], -(b * sn[i & 3]));
        x[2 * i + 1] = fmaf(b, cs[i & 3], a * sn[i & 3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(0xffffffffu, x[e], partner);
        if (turns) x[e] = fmaf(x[e], cs[e], o * sn[e]);
      }
    }
  }
};

// the sum over the LANES lanes of a row
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <class T>
__device__ __forceinline__ void load_weight(float (&w)[8], const void* p, int c, bool in) {
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 1.0f;
  if (!p || !in) return;
  Raw<T> r;
  r.load(static_cast<const T*>(p) + c);
  r.get(w);
}

template <class T, int LANES, bool INTER, bool STORE>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int kHeads = 32 / LANES;  // of a pass
  const int lane = threadIdx.x & 31, sub = lane / LANES, c = (lane & (LANES - 1)) * 8;
  const bool col = c < A.dim;
  Turn<INTER> turn;
  turn.place(A.rot, col ? c : A.dim, lane);
  grid_begin();
  float qw[8], kw[8];
  if (A.norm) {
    load_weight<T>(qw, A.qw, c, col);
    load_weight<T>(kw, A.kw, c, col);
  }
  const float inv_dim = 1.0f / (float)A.dim;
  const int rows = A.heads + A.kv_heads * (STORE ? 2 : 1);
  const int passes = (rows + kHeads - 1) / kHeads, mine = (passes + A.split - 1) / A.split;
  const int tasks = A.tokens * A.split, warps = (int)(gridDim.x * (kRopeThreads / 32));
  for (int task = (int)(blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5)); task < tasks; task += warps) {
    const int t = A.split == 1 ? task : task / A.split;
    const int p0 = (task - t * A.split) * mine, p1 = p0 + mine < passes ? p0 + mine : passes;
    if (p0 >= p1) continue;
    const T* const q = static_cast<const T*>(A.q.p) + t * A.q.token + c;
    const T* const k = static_cast<const T*>(A.k.p) + t * A.k.token + c;
    const T* const v = STORE ? static_cast<const T*>(A.v.p) + t * A.v.token + c : nullptr;
    T* const qo = static_cast<T*>(A.qo.p) + t * A.qo.token + c;
    T* const ko = STORE ? nullptr : static_cast<T*>(A.ko.p) + t * A.ko.token + c;
    int64_t at = -1;  // of the token in the pools
    bool ready = false;
#pragma unroll 1
    for (int p = p0; p < p1; p += kRopeFlight) {
      Raw<T> x[kRopeFlight];
#pragma unroll
      for (int i = 0; i < kRopeFlight; ++i) {
        const int u = (p + i) * kHeads + sub;
        x[i].zero();
        if (p + i >= p1 || u >= rows || !col) continue;
        x[i].load(u < A.heads ? q + u * A.q.head
                  : !STORE || u < A.heads + A.kv_heads ? k + (u - A.heads) * A.k.head
                                                       : v + (u - A.heads - A.kv_heads) * A.v.head);
      }
      if (!ready) {  // behind the first rows' loads
        ready = true;
        turn.at(A, ld_plain(A.positions + t), c, 1.0f);
        if (STORE) {
          const int64_t slot = ld_plain(A.slots + t), page = slot >> A.page_log2;
          if (slot >= 0 && page >= A.c.pages) raise_error(A.err, TP3D_EPAGES);
          if (slot >= 0 && page < A.c.pages)
            at = page * A.c.page_stride + (slot & ((1 << A.page_log2) - 1)) * A.c.token_stride + c;
        }
      }
#pragma unroll
      for (int i = 0; i < kRopeFlight; ++i) {
        if (p + i >= p1) break;
        const int u = (p + i) * kHeads + sub;
        const bool value = STORE && u >= A.heads + A.kv_heads;
        // passes of value rows alone are copied as they are
        if (!STORE || (p + i) * kHeads < A.heads + A.kv_heads) {
          float y[8];
          x[i].get(y);
          if (A.norm) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(y[e], y[e], s);
            s = rsqrtf(fmaf(row_sum<LANES>(s), inv_dim, A.eps));
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * s * (u < A.heads ? qw[e] : kw[e]);
          }
          turn.apply(y);
          if (!value) x[i].set(y);
        }
        if (u >= rows || !col) continue;
        if (u < A.heads) x[i].store(qo + u * A.qo.head);
        else if (!STORE) x[i].store(ko + (u - A.heads) * A.ko.head);
        else if (at >= 0)
          x[i].store(static_cast<T*>(value ? A.c.v : A.c.k) + at +
                     (u - A.heads - (value ? A.kv_heads : 0)) * A.c.head_stride);
      }
    }
  }
}

// Backward: g = R(p)^T dy; with the norm dx = s (w g - x s^2 mean(w g x)) and the
// weights' gradients, the sums of g x s, kept in registers over a warp's tokens,
// joined warp by warp in shared memory and CTA by CTA in the workspace, in a
// fixed order; the last CTA to arrive adds the CTAs' parts.
template <class T, int LANES, bool INTER>
__global__ void __launch_bounds__(kBackThreads, 1) rope_back_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int kHeads = 32 / LANES, kWarps = kBackThreads / 32;
  extern __shared__ float sums[];  // [warp][q or k][dim]
  __shared__ int last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LANES, c = (lane & (LANES - 1)) * 8;
  const bool col = c < A.dim;
  Turn<INTER> turn;
  turn.place(A.rot, col ? c : A.dim, lane);
  grid_begin();
  float qw[8], kw[8], sq[8], sk[8];
  if (A.norm) {
    load_weight<T>(qw, A.qw, c, col);
    load_weight<T>(kw, A.kw, c, col);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sq[e] = sk[e] = 0.0f;
  const float inv_dim = 1.0f / (float)A.dim;
  const int rows = A.heads + A.kv_heads;
  const int passes = (rows + kHeads - 1) / kHeads, mine = (passes + A.split - 1) / A.split;
  const int tasks = A.tokens * A.split, warps = (int)gridDim.x * kWarps;
  // consecutive tasks to different CTAs: few tasks fill the SMs evenly
  for (int task = warp * (int)gridDim.x + (int)blockIdx.x; task < tasks; task += warps) {
    const int t = A.split == 1 ? task : task / A.split;
    const int p0 = (task - t * A.split) * mine, p1 = p0 + mine < passes ? p0 + mine : passes;
    if (p0 >= p1) continue;
    const T* const q = static_cast<const T*>(A.q.p) + t * A.q.token + c;
    const T* const k = static_cast<const T*>(A.k.p) + t * A.k.token + c;
    const T* const dq = static_cast<const T*>(A.dq.p) + t * A.dq.token + c;
    const T* const dk = static_cast<const T*>(A.dk.p) + t * A.dk.token + c;
    T* const qo = static_cast<T*>(A.qo.p) + t * A.qo.token + c;
    T* const ko = static_cast<T*>(A.ko.p) + t * A.ko.token + c;
    bool ready = false;
    constexpr int kFlight = kRopeFlight / 2;  // of x and of dy each
#pragma unroll 1
    for (int p = p0; p < p1; p += kFlight) {
      Raw<T> x[kFlight], dy[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int u = (p + i) * kHeads + sub;
        x[i].zero();
        dy[i].zero();
        if (p + i >= p1 || u >= rows || !col) continue;
        dy[i].load(u < A.heads ? dq + u * A.dq.head : dk + (u - A.heads) * A.dk.head);
        if (A.norm) x[i].load(u < A.heads ? q + u * A.q.head : k + (u - A.heads) * A.k.head);
      }
      if (!ready) {
        ready = true;
        turn.at(A, ld_plain(A.positions + t), c, -1.0f);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        if (p + i >= p1) break;
        const int u = (p + i) * kHeads + sub;
        float g[8];
        dy[i].get(g);
        turn.apply(g);
        if (A.norm) {
          float y[8], s = 0.0f, dot = 0.0f;
          x[i].get(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(y[e], y[e], s);
          s = rsqrtf(fmaf(row_sum<LANES>(s), inv_dim, A.eps));
          const bool is_q = u < A.heads, is_k = !is_q && u < rows;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] *= s;
            const float dw = g[e] * y[e];
            sq[e] += is_q ? dw : 0.0f;
            sk[e] += is_k ? dw : 0.0f;
            const float w = is_q ? qw[e] : kw[e];
            dot = fmaf(dw, w, dot);
            g[e] *= w;
          }
          dot = row_sum<LANES>(dot) * inv_dim;
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = s * fmaf(-y[e], dot, g[e]);
        }
        dy[i].set(g);
        if (u >= rows || !col) continue;
        if (u < A.heads) dy[i].store(qo + u * A.qo.head);
        else dy[i].store(ko + (u - A.heads) * A.ko.head);
      }
    }
  }
  if (!A.parts) return;
  const int width = 2 * A.dim;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
      sq[e] += __shfl_xor_sync(0xffffffffu, sq[e], o);
      sk[e] += __shfl_xor_sync(0xffffffffu, sk[e], o);
    }
    if (sub == 0 && col) {
      sums[warp * width + c + e] = sq[e];
      sums[warp * width + A.dim + c + e] = sk[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += kBackThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w * width + i];
    __stcg(A.parts + (size_t)blockIdx.x * width + i, s);
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicInc(A.arrivals, gridDim.x - 1) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // four columns to a thread; group g of `groups` adds every groups-th part, then the groups are added
  const int quads = width / 4, fit = kBackThreads / quads, groups = fit < kWarps ? fit : kWarps;  // (the size of `sums`)
  const int g = (int)threadIdx.x / quads, at = (int)threadIdx.x - g * quads;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (g < groups) {
#pragma unroll 8
    for (int b = g; b < (int)gridDim.x; b += groups) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(A.parts + (size_t)b * width) + at);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    reinterpret_cast<float4*>(sums)[g * quads + at] = s;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += kBackThreads) {
    float x = 0.0f;
    for (int j = 0; j < groups; ++j) x += sums[j * width + i];
    T* const to = static_cast<T*>(i < A.dim ? A.dqw : A.dkw);
    if (to) to[i < A.dim ? i : i - A.dim] = (T)x;
  }
}

// zeros, where there are no tokens to sum over
template <class T>
__global__ void rope_zero_kernel(T* q, T* k, int dim) {
  grid_begin();
  if ((int)threadIdx.x >= dim) return;
  if (q) q[threadIdx.x] = (T)0.0f;
  if (k) k[threadIdx.x] = (T)0.0f;
}

// ------------------------------------------------------------------ host side
int esize(int dtype) { return dtype == TP3D_BF16 ? 2 : 4; }

tp3d_status check_rope(const tp3d_rope* r) {
  if (!r) return TP3D_EINVAL;
  if (r->dtype != TP3D_BF16 && r->dtype != TP3D_F32) return TP3D_EDTYPE;
  if (r->head_dim < 1 || r->rotary_dim < 0 || r->norm < 0 || r->norm > 1 || r->interleaved < 0 || r->interleaved > 1)
    return TP3D_EINVAL;
  if (!isfinite(r->magnitude) || (r->norm && (!isfinite(r->eps) || r->eps < 0.0f))) return TP3D_EINVAL;
  if (r->rotary_dim > r->head_dim) return TP3D_ESHAPE;
  if (r->head_dim % 8 || r->head_dim > 256 || r->rotary_dim % 16) return TP3D_EUNSUPPORTED;
  if (r->rotary_dim && !r->turns) return TP3D_EINVAL;
  if (!aligned(r->turns, 8) || !aligned16(r->q_weight) || !aligned16(r->k_weight)) return TP3D_EALIGN;
  return TP3D_OK;
}

// (token, head) rows on the host: what the checks need of them
struct Rows {
  const void* p;
  int64_t token, head;
  int heads;
};
Rows rows(const void* p, tp3d_row_strides s, int heads) { return Rows{p, s.token_stride, s.head_stride, heads}; }

tp3d_status check_rows(const Rows& r, int elem_bytes) {
  if (!r.p || r.token < 1 || r.head < 1) return TP3D_EINVAL;
  if ((r.token | r.head) >> 39) return TP3D_EUNSUPPORTED;
  if (!aligned16(r.p) || r.token * elem_bytes % 16 || r.head * elem_bytes % 16) return TP3D_EALIGN;
  return TP3D_OK;
}
size_t rows_bytes(const Rows& r, int64_t tokens, int dim, int elem_bytes) {
  return extent(1, 0, tokens, r.token, r.heads, r.head, dim, elem_bytes);
}
bool rows_clash(const Rows& a, const Rows& b, int64_t tokens, int dim, int elem_bytes) {
  if (!overlaps(a.p, rows_bytes(a, tokens, dim, elem_bytes), b.p, rows_bytes(b, tokens, dim, elem_bytes))) return false;
  if (a.token != b.token) return true;
  // slices of the same rows: what one token's part of each takes up, modulo the step from token to token
  const uint64_t step = (uint64_t)a.token * elem_bytes;
  const uint64_t na = ((uint64_t)(a.heads - 1) * a.head + dim) * elem_bytes;
  const uint64_t nb = ((uint64_t)(b.heads - 1) * b.head + dim) * elem_bytes;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t off = y >= x ? (y - x) % step : (step - (x - y) % step) % step;
  return na > step || nb > step || off < na || off + nb > step;
}
bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.token == b.token && a.head == b.head; }

// An array of `n` bytes against the rows that are written.
bool range_clash(const Rows& r, int64_t tokens, int dim, int elem_bytes, const void* p, size_t n) {
  return overlaps(r.p, rows_bytes(r, tokens, dim, elem_bytes), p, n);
}
bool rope_clash(const Rows& r, int64_t tokens, const tp3d_rope& R, int elem_bytes, const int32_t* positions) {
  const size_t wb = (size_t)R.head_dim * elem_bytes;
  return range_clash(r, tokens, R.head_dim, elem_bytes, positions, (size_t)tokens * 4) ||
         (R.rotary_dim && range_clash(r, tokens, R.head_dim, elem_bytes, R.turns, (size_t)R.rotary_dim * 4)) ||
         (R.norm && (range_clash(r, tokens, R.head_dim, elem_bytes, R.q_weight, wb) ||
                     range_clash(r, tokens, R.head_dim, elem_bytes, R.k_weight, wb)));
}

RopeArgs rope_args(const tp3d_rope& R, int64_t tokens, int heads, int kv_heads, const int32_t* positions) {
  RopeArgs A{};
  A.tokens = (int32_t)tokens;
  A.heads = heads;
  A.kv_heads = kv_heads;
  A.dim = R.head_dim;
  A.rot = R.rotary_dim;
  A.norm = R.norm;
  A.eps = R.eps;
  A.magnitude = R.magnitude;
  A.turns = R.turns;
  A.qw = R.norm ? R.q_weight : nullptr;
  A.kw = R.norm ? R.k_weight : nullptr;
  A.positions = positions;
  return A;
}
RowsIn in(const Rows& r) { return RowsIn{r.p, r.token, r.head}; }
RowsOut out(const Rows& r) { return RowsOut{const_cast<void*>(r.p), r.token, r.head}; }

int lanes_of(int dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// Warps for each token: one, unless the tokens leave SMs without `per_sm` warps; then as many as
// there are passes over its heads.
int split_of(const tp3d_ctx* ctx, int64_t tokens, int rows, int lanes, int per_sm) {
  const int64_t passes = (rows + 32 / lanes - 1) / (32 / lanes), want = (int64_t)ctx->num_sms * per_sm;
  const int64_t s = (want + tokens - 1) / tokens;
  return (int)(s < 1 ? 1 : s < passes ? s : passes);
}

template <class T, int LANES, bool STORE>
tp3d_status launch_rope_lanes(const tp3d_ctx* ctx, RopeArgs& A, int interleaved, cudaStream_t s) {
  A.split = split_of(ctx, A.tokens, A.heads + A.kv_heads * (STORE ? 2 : 1), LANES, 16);
  const int64_t ctas = ((int64_t)A.tokens * A.split + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const unsigned grid = (unsigned)(ctas < ctx->num_sms * 2 ? ctas : ctx->num_sms * 2);
  return interleaved ? launch_dependent(rope_kernel<T, LANES, true, STORE>, grid, kRopeThreads, 0, s, A)
                     : launch_dependent(rope_kernel<T, LANES, false, STORE>, grid, kRopeThreads, 0, s, A);
}
template <class T, bool STORE>
tp3d_status launch_rope(const tp3d_ctx* ctx, RopeArgs& A, int interleaved, cudaStream_t s) {
  const int lanes = lanes_of(A.dim);
  if (lanes == 8) return launch_rope_lanes<T, 8, STORE>(ctx, A, interleaved, s);
  if (STORE || lanes == 16) return launch_rope_lanes<T, 16, STORE>(ctx, A, interleaved, s);  // (a cache's heads: 64 or 128)
  return launch_rope_lanes<T, STORE ? 16 : 32, STORE>(ctx, A, interleaved, s);
}

template <class T, int LANES>
tp3d_status launch_back_lanes(const tp3d_ctx* ctx, RopeArgs& A, int interleaved, cudaStream_t s) {
  A.split = split_of(ctx, A.tokens, A.heads + A.kv_heads, LANES, kBackThreads / 32);
  const int64_t tasks = (int64_t)A.tokens * A.split;
  const unsigned grid = (unsigned)(tasks < ctx->num_sms ? tasks : ctx->num_sms);
  const size_t smem = A.parts ? (size_t)(kBackThreads / 32) * 2 * A.dim * sizeof(float) : 0;  // 32 KiB at most
  return interleaved ? launch_dependent(rope_back_kernel<T, LANES, true>, grid, kBackThreads, smem, s, A)
                     : launch_dependent(rope_back_kernel<T, LANES, false>, grid, kBackThreads, smem, s, A);
}
template <class T>
tp3d_status launch_back(const tp3d_ctx* ctx, RopeArgs& A, int interleaved, cudaStream_t s) {
  if (A.tokens == 0)
    return launch_dependent(rope_zero_kernel<T>, 1, 256, 0, s, static_cast<T*>(A.dqw), static_cast<T*>(A.dkw), A.dim);
  switch (lanes_of(A.dim)) {
    case 8: return launch_back_lanes<T, 8>(ctx, A, interleaved, s);
    case 16: return launch_back_lanes<T, 16>(ctx, A, interleaved, s);
    default: return launch_back_lanes<T, 32>(ctx, A, interleaved, s);
  }
}

// most tokens x warps of a token, and rows: in 32 bits
tp3d_status check_counts(int64_t tokens, int heads, int kv_heads) {
  if (tokens < 0 || heads < 1 || kv_heads < 1) return TP3D_EINVAL;
  if (tokens > kPagedMaxTokens || heads > 65536 || kv_heads > 65536) return TP3D_EUNSUPPORTED;
  return TP3D_OK;
}

}  // namespace

}  // namespace tp3d

using namespace tp3d;

extern "C" {

tp3d_status tp3d_qk_rope(tp3d_ctx* ctx, const tp3d_rope* rope, int64_t tokens, int heads, int kv_heads, const void* Q,
                         tp3d_row_strides q_strides, const void* K, tp3d_row_strides k_strides,
                         const int32_t* positions, void* Q_out, tp3d_row_strides qo_strides, void* K_out,
                         tp3d_row_strides ko_strides, void* stream) {
  if (!ctx) return TP3D_EINVAL;
  TP3D_TRY(check_rope(rope));
  TP3D_TRY(check_counts(tokens, heads, kv_heads));
  if (tokens == 0) return TP3D_OK;
  const int es = esize(rope->dtype), d = rope->head_dim;
  const Rows q = rows(Q, q_strides, heads), k = rows(K, k_strides, kv_heads);
  const Rows qo = rows(Q_out, qo_strides, heads), ko = rows(K_out, ko_strides, kv_heads);
  for (const Rows* r : {&q, &k, &qo, &ko}) TP3D_TRY(check_rows(*r, es));
  if (!positions) return TP3D_EINVAL;
  if (!aligned(positions, 4)) return TP3D_EALIGN;
  if ((!same_rows(q, qo) && rows_clash(qo, q, tokens, d, es)) || (!same_rows(k, ko) && rows_clash(ko, k, tokens, d, es)) ||
      rows_clash(qo, k, tokens, d, es) || rows_clash(ko, q, tokens, d, es) || rows_clash(qo, ko, tokens, d, es) ||
      rope_clash(qo, tokens, *rope, es, positions) || rope_clash(ko, tokens, *rope, es, positions))
    return TP3D_EOVERLAP;
  RopeArgs A = rope_args(*rope, tokens, heads, kv_heads, positions);
  A.q = in(q);
  A.k = in(k);
  A.qo = out(qo);
  A.ko = out(ko);
  A.err = ctx->d_err;
  const cudaStream_t s = as_stream(stream);
  return rope->dtype == TP3D_BF16 ? launch_rope<__nv_bfloat16, false>(ctx, A, rope->interleaved, s)
                                  : launch_rope<float, false>(ctx, A, rope->interleaved, s);
}

size_t tp3d_qk_rope_bwd_workspace_bytes(tp3d_ctx* ctx, const tp3d_rope* rope) {
  if (!ctx || check_rope(rope) != TP3D_OK) return 0;
  return (size_t)ctx->num_sms * 2 * rope->head_dim * sizeof(float);
}

tp3d_status tp3d_qk_rope_bwd(tp3d_ctx* ctx, const tp3d_rope* rope, int64_t tokens, int heads, int kv_heads,
                             const void* Q, tp3d_row_strides q_strides, const void* K, tp3d_row_strides k_strides,
                             const int32_t* positions, const void* dQ_out, tp3d_row_strides dqo_strides,
                             const void* dK_out, tp3d_row_strides dko_strides, void* dQ, tp3d_row_strides dq_strides,
                             void* dK, tp3d_row_strides dk_strides, void* dq_weight, void* dk_weight, void* workspace,
                             void* stream) {
  if (!ctx) return TP3D_EINVAL;
  TP3D_TRY(check_rope(rope));
  TP3D_TRY(check_counts(tokens, heads, kv_heads));
  const bool sums = dq_weight || dk_weight;
  if (sums && !rope->norm) return TP3D_EINVAL;
  if (sums && !workspace) return TP3D_EINVAL;
  if (!aligned16(dq_weight) || !aligned16(dk_weight) || (sums && !aligned(workspace, 256))) return TP3D_EALIGN;
  const int es = esize(rope->dtype), d = rope->head_dim;
  const size_t wb = (size_t)d * es, ws = sums ? tp3d_qk_rope_bwd_workspace_bytes(ctx, rope) : 0;
  const Range sum_out[] = {{dq_weight, wb}, {dk_weight, wb}, {workspace, ws}};
  const Range sum_in[] = {{rope->turns, (size_t)rope->rotary_dim * 4}, {rope->norm ? rope->q_weight : nullptr, wb},
                          {rope->norm ? rope->k_weight : nullptr, wb}};
  if (clash(sum_out, sum_in)) return TP3D_EOVERLAP;
  const Rows q = rows(Q, q_strides, heads), k = rows(K, k_strides, kv_heads);
  const Rows gq = rows(dQ_out, dqo_strides, heads), gk = rows(dK_out, dko_strides, kv_heads);
  const Rows dq = rows(dQ, dq_strides, heads), dk = rows(dK, dk_strides, kv_heads);
  if (tokens > 0) {
    if (rope->norm)
      for (const Rows* r : {&q, &k}) TP3D_TRY(check_rows(*r, es));
    for (const Rows* r : {&gq, &gk, &dq, &dk}) TP3D_TRY(check_rows(*r, es));
    if (!positions) return TP3D_EINVAL;
    if (!aligned(positions, 4)) return TP3D_EALIGN;
    if ((!same_rows(dq, gq) && rows_clash(dq, gq, tokens, d, es)) ||
        (!same_rows(dk, gk) && rows_clash(dk, gk, tokens, d, es)) || rows_clash(dq, gk, tokens, d, es) ||
        rows_clash(dk, gq, tokens, d, es) || rows_clash(dq, dk, tokens, d, es))
      return TP3D_EOVERLAP;
    for (const Rows* r : {&dq, &dk}) {
      if (rope->norm && (rows_clash(*r, q, tokens, d, es) || rows_clash(*r, k, tokens, d, es))) return TP3D_EOVERLAP;
      if (rope_clash(*r, tokens, *rope, es, positions)) return TP3D_EOVERLAP;
    }
    for (const Range& o : sum_out) {
      if (overlaps(o.p, o.n, positions, (size_t)tokens * 4)) return TP3D_EOVERLAP;
      for (const Rows* r : {&q, &k, &gq, &gk, &dq, &dk})
        if ((rope->norm || (r != &q && r != &k)) && range_clash(*r, tokens, d, es, o.p, o.n)) return TP3D_EOVERLAP;
    }
  } else if (!sums) {
    return TP3D_OK;
  }
  RopeArgs A = rope_args(*rope, tokens, heads, kv_heads, positions);
  A.q = in(q);
  A.k = in(k);
  A.dq = in(gq);
  A.dk = in(gk);
  A.qo = out(dq);
  A.ko = out(dk);
  A.dqw = dq_weight;
  A.dkw = dk_weight;
  A.parts = sums ? static_cast<float*>(workspace) : nullptr;
  A.arrivals = ctx->d_paged + kRopeCounter;
  const cudaStream_t s = as_stream(stream);
  return rope->dtype == TP3D_BF16 ? launch_back<__nv_bfloat16>(ctx, A, rope->interleaved, s)
                                  : launch_back<float>(ctx, A, rope->interleaved, s);
}

tp3d_status tp3d_paged_rope_store(tp3d_ctx* ctx, const tp3d_rope* rope, const tp3d_kv_cache* cache, int64_t tokens,
                                  int heads, const void* Q, tp3d_row_strides q_strides, const void* K,
                                  tp3d_row_strides k_strides, const void* V, tp3d_row_strides v_strides,
                                  const int32_t* positions, const int64_t* slots, void* Q_out,
                                  tp3d_row_strides qo_strides, void* stream) {
  if (!ctx) return TP3D_EINVAL;
  TP3D_TRY(check_cache(cache));
  TP3D_TRY(check_rope(rope));
  if (rope->dtype != cache->dtype) return TP3D_EDTYPE;
  if (rope->head_dim != cache->head_dim) return TP3D_ESHAPE;
  TP3D_TRY(check_counts(tokens, heads, cache->kv_heads));
  if (tokens == 0) return TP3D_OK;
  const int es = esize(rope->dtype), d = rope->head_dim;
  const Rows q = rows(Q, q_strides, heads), qo = rows(Q_out, qo_strides, heads);
  const Rows k = rows(K, k_strides, cache->kv_heads), v = rows(V, v_strides, cache->kv_heads);
  for (const Rows* r : {&q, &k, &v, &qo}) TP3D_TRY(check_rows(*r, es));
  if (!positions || !slots) return TP3D_EINVAL;
  if (!aligned(positions, 4) || !aligned(slots, 8)) return TP3D_EALIGN;
  if ((!same_rows(q, qo) && rows_clash(qo, q, tokens, d, es)) || rows_clash(qo, k, tokens, d, es) ||
      rows_clash(qo, v, tokens, d, es) || rope_clash(qo, tokens, *rope, es, positions) ||
      range_clash(qo, tokens, d, es, slots, (size_t)tokens * 8))
    return TP3D_EOVERLAP;
  // the two pools may share one allocation (interleaved pages), so only the others are checked against them
  const size_t cb = cache_bytes(*cache), wb = (size_t)d * es;
  for (const void* pool : {cache->k, cache->v}) {
    for (const Rows* r : {&q, &k, &v, &qo})
      if (range_clash(*r, tokens, d, es, pool, cb)) return TP3D_EOVERLAP;
    if (overlaps(pool, cb, positions, (size_t)tokens * 4) || overlaps(pool, cb, slots, (size_t)tokens * 8) ||
        overlaps(pool, cb, rope->turns, (size_t)rope->rotary_dim * 4) ||
        (rope->norm && (overlaps(pool, cb, rope->q_weight, wb) || overlaps(pool, cb, rope->k_weight, wb))))
      return TP3D_EOVERLAP;
  }
  RopeArgs A = rope_args(*rope, tokens, heads, cache->kv_heads, positions);
  A.q = in(q);
  A.k = in(k);
  A.v = in(v);
  A.qo = out(qo);
  A.c = *cache;
  A.page_log2 = page_log2(cache->page);
  A.slots = slots;
  A.err = ctx->d_err;
  return launch_rope<__nv_bfloat16, true>(ctx, A, rope->interleaved, as_stream(stream));
}

}  // extern "C"
