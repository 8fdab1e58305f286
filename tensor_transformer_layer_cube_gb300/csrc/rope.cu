// rope.cu - the norm of query and key heads with the rotation by position:
// forward, backward, and the form that writes keys and values to the paged
// cache (include/tp3d_rope.h, tp3d_paged_rope_store of include/tp3d_paged.h).
//
// Row x of one head at position p: n = x s w with s = 1 / sqrt(mean x^2 + eps),
// y = R(p) n.  R turns pairs of columns by p f_j; with the frequency as a 64-bit
// fraction F of a turn, the angle is p F mod 2^64: an integer product that
// drops whole turns by itself, rounded to fp32 when whole quarter turns are off.
//
// Every element is read once and written once, so HBM bounds many tokens and
// latency few; instructions come close behind, so a pass is made of few.  A row
// lies on LANES neighbouring lanes, each with two groups of four columns,
// rotary_dim / 2 apart, so that both columns of a pair are one lane's and
// neighbouring lanes' groups are neighbours.  A warp's pass takes the same head
// of 32 / LANES tokens, and its passes go over their query heads, then their key
// heads (then their values).  With x' the other column of each column's pair, a
// row of y is
//   y = s (A x + B x'),  A = m w cos,  B = -+ m w' sin,
// with the angles computed once for a token and A and B for its heads of one
// kind.  Passes are loaded several ahead into a ring in shared memory that each
// lane fills and reads by itself (4 KiB a warp, no barrier), over the ends of
// tokens.  All passes in a row are cut into equal ranges, one for each warp.
//
// Measured, of a stream of calls: 16385 tokens of 32 heads of 128 on 8, with the
// store (403 MB) 69.5 us, 0.85 of the copy rate; 4095 tokens of 12 heads of 96 on
// 4 in fp32, half of each turned (50 MB) 12.0 us, 0.62; 64 tokens of 16 heads of
// 128 with the store 7.5 us, of which the GPU's part is 3.8.  A pass is 102
// instructions; with rows of one token in a pass, their pairs on different lanes
// and the angles by CUDA's function it was 195, and the times 95.8, 13.4 and 9.9.
#include <math.h>

#include "paged.cuh"

namespace tp3d {

namespace {

constexpr int kRopeThreads = 256, kBackThreads = 512;
constexpr int kRingBytes = 4096;  // of a warp

struct RowsIn {
  const void* p;
  int64_t token, head;
};
struct RowsOut {
  void* p;
  int64_t token, head;
};

struct RopeArgs {
  int32_t tokens, heads, kv_heads, dim, rot, norm;
  int32_t range;  // passes of a warp
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

__device__ __forceinline__ void cp_async(uint32_t dst, const __nv_bfloat16* src) {  // four columns
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async(uint32_t dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A lane's eight columns of a row, as pairs of fp32: two groups of four.
template <class T>
struct Row;
template <>
struct Row<__nv_bfloat16> {
  static constexpr uint32_t kBytes = 16, kGroup = 8;  // of a lane in the ring, and from its first group to its second
  uint4 w;
  __device__ __forceinline__ void read(uint32_t at) { w = ld_shared4(at); }
  __device__ __forceinline__ void get(f32x2 (&x)[4]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pk2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void set(const f32x2 (&x)[4]) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      upk2(x[i], a, b);
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      v[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    w = make_uint4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ void write(__nv_bfloat16* p, int second) const {
    *reinterpret_cast<uint2*>(p) = make_uint2(w.x, w.y);
    *reinterpret_cast<uint2*>(p + second) = make_uint2(w.z, w.w);
  }
};
template <>
struct Row<float> {
  static constexpr uint32_t kBytes = 32, kGroup = 512;  // the second groups of all lanes behind the first ones
  uint4 w, v;
  __device__ __forceinline__ void read(uint32_t at) {
    w = ld_shared4(at);
    v = ld_shared4(at + kGroup);
  }
  __device__ __forceinline__ void get(f32x2 (&x)[4]) const {
    x[0] = pk2(__uint_as_float(w.x), __uint_as_float(w.y));
    x[1] = pk2(__uint_as_float(w.z), __uint_as_float(w.w));
    x[2] = pk2(__uint_as_float(v.x), __uint_as_float(v.y));
    x[3] = pk2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ void set(const f32x2 (&x)[4]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) upk2(x[i], f[2 * i], f[2 * i + 1]);
    w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    v = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
  __device__ __forceinline__ void write(float* p, int second) const {
    *reinterpret_cast<uint4*>(p) = w;
    *reinterpret_cast<uint4*>(p + second) = v;
  }
};

// Sine and cosine of an angle in units of 2^-64 turns: a whole number of quarter
// turns off, what is left (an eighth of a turn at most) goes through the Taylor
// series, whose next terms are below 2^-29 and 2^-33.  Either is off by 5 2^-24 of
// itself at most, small ones too: a slow pair's sine is as small as its angle, and
// stands alone where the pair's other column is small.  (The upper 32 bits alone
// leave 5.6e-6 off by 2.5e-4 of itself.  4095 tokens in fp32 12.0 us, with those alone
// 11.9, with one conversion of all 64 bits 12.4.)
__device__ __forceinline__ void sincos_of(uint64_t turn, float& s, float& c) {
  const uint32_t hi = (uint32_t)(turn >> 32), lo = (uint32_t)turn, q = (hi + 0x20000000u) >> 30;
  // the halves as signed numbers, so that neither takes much of the other away; by 2 pi / 2^32 and 2 pi / 2^64
  const float t = fmaf((float)(int32_t)(hi - (q << 30) + (lo >> 31)), 1.4629180792671596e-9f,
                       (float)(int32_t)lo * 3.4061215800865545e-19f);
  const float x = t * t;
  const float a = fmaf(t * x, fmaf(x, fmaf(x, fmaf(x, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), t);
  const float b = fmaf(
      x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const float y = q & 1 ? b : a, z = q & 1 ? a : b;
  s = __uint_as_float(__float_as_uint(y) ^ (q & 2) << 30);
  c = __uint_as_float(__float_as_uint(z) ^ ((q + 1) & 2) << 30);
}

// A lane's columns [c, c + 4) and [c + second, + 4), and their rotation.
template <bool INTER>
struct Turn {
  int c, second;
  bool in, turned;     // these are columns of the row; they are turned
  float cs[4], sn[4];  // cosines and sines of the lane's four pairs, times the magnitude
  __device__ __forceinline__ void place(const RopeArgs& A, int l) {
    turned = 8 * l < A.rot;
    in = 8 * l < A.dim;
    c = turned ? 4 * l : in ? A.rot / 2 + 4 * l : 0;
    second = turned ? A.rot / 2 : in ? (A.dim - A.rot) / 2 : 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = 1.0f, sn[e] = 0.0f;
  }
  __device__ __forceinline__ void at(const RopeArgs& A, int pos) {
    if (!turned) return;
    const uint64_t* const turns = A.turns + (INTER ? c / 2 : c);
    const int hop = INTER ? A.rot / 4 - 2 : 0;  // from the first group's pairs to the second's
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sincos_of((uint64_t)(int64_t)pos * ld_plain(turns + (e < 2 ? e : e + hop)), sn[e], cs[e]);
      cs[e] *= A.magnitude;
      sn[e] *= A.magnitude;
    }
  }
  // The factors of x and x' for weights w; back: of the transposed rotation (and no weights).
  __device__ __forceinline__ void factors(const float (&w)[8], bool back, f32x2 (&a)[4], f32x2 (&b)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 2 * i;
      if (INTER) {
        const float s = back ? -sn[i] : sn[i];
        a[i] = pk2(cs[i] * w[e], cs[i] * w[e + 1]);
        b[i] = pk2(-s * w[e + 1], s * w[e]);
      } else {
        const int o = e ^ 4, p = e & 3;  // the pair's other columns; its place among the four
        const bool minus = (e < 4) != back;
        a[i] = pk2(cs[p] * w[e], cs[p + 1] * w[e + 1]);
        b[i] = pk2((minus ? -sn[p] : sn[p]) * w[o], (minus ? -sn[p + 1] : sn[p + 1]) * w[o + 1]);
      }
      if (!turned) b[i] = 0;
    }
  }
  // x = a x + b x'.  `all`: every lane's columns are turned; else those that are not only take their weight, since
  // 0 times an x' that is not finite is none.
  __device__ __forceinline__ void apply(f32x2 (&x)[4], const f32x2 (&a)[4], const f32x2 (&b)[4], bool all) const {
    f32x2 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (INTER) {
        float lo, hi;
        upk2(x[i], lo, hi);
        o[i] = pk2(hi, lo);
      } else {
        o[i] = x[i ^ 2];
      }
    }
    if (all) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = fma2(x[i], a[i], mul2(o[i], b[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = turned ? fma2(x[i], a[i], mul2(o[i], b[i])) : mul2(x[i], a[i]);
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
// The sums over the LANES lanes of a row, of two values: from the first step on
// even lanes go on with a, odd ones with b.
template <int LANES>
__device__ __forceinline__ void row_sums(float& a, float& b, int lane) {
  const bool odd = lane & 1;
  float v = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
#pragma unroll
  for (int o = 2; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const float u = __shfl_xor_sync(0xffffffffu, v, 1);
  a = odd ? u : v;
  b = odd ? v : u;
}
__device__ __forceinline__ float sum_of(f32x2 v) {
  float a, b;
  upk2(v, a, b);
  return a + b;
}
// 1 / sqrt(mean x^2 + eps) of a row
template <int LANES>
__device__ __forceinline__ float inverse_rms(float eps, const f32x2 (&x)[4], float inv_dim) {
  f32x2 q = mul2(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) q = fma2(x[i], x[i], q);
  return rsqrtf(fmaf(row_sum<LANES>(sum_of(q)), inv_dim, eps));
}

// the weights in shared memory: query heads', then key heads' (kWeights columns each, those past the heads 1)
constexpr int kWeights = 256;
template <class T>
__device__ __forceinline__ void fill_weights(const RopeArgs& A, float* w) {
  for (int i = threadIdx.x; i < 2 * kWeights; i += blockDim.x) {
    const T* const p = static_cast<const T*>(i < kWeights ? A.qw : A.kw);
    const int c = i & (kWeights - 1);
    w[i] = p && c < A.dim ? (float)ld_plain(p + c) : 1.0f;
  }
  __syncthreads();
}
__device__ __forceinline__ void columns_of(const float* w, int c, int second, float (&x)[8]) {
  const float4 v = *reinterpret_cast<const float4*>(w + c), u = *reinterpret_cast<const float4*>(w + c + second);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w, x[4] = u.x, x[5] = u.y, x[6] = u.z, x[7] = u.w;
}

// What a warp goes over: `range` passes from its first on, pass p of the `all` of
// each group of neighbouring tokens, group by group.  The first nq of a group are
// query heads, the next nk key heads, the others values: one kind after the other.
struct Walk {
  int nq, nk, all;
  int group, p, rest;  // rest: passes of the range from this one on
  __device__ __forceinline__ void begin(const RopeArgs& A, int kinds, int tokens, int warp) {
    nq = A.heads;
    nk = A.kv_heads;
    all = nq + (kinds - 1) * nk;
    const int64_t groups = ((int64_t)A.tokens + tokens - 1) / tokens;
    const int64_t first = (int64_t)warp * A.range, left = groups * all - first;
    rest = left < A.range ? left < 0 ? 0 : (int)left : A.range;
    group = (int)(first / all);
    p = (int)(first - (int64_t)group * all);
  }
  __device__ __forceinline__ int kind() const { return p < nq ? 0 : p < nq + nk ? 1 : 2; }
  // the head of pass p, and the passes of its kind from it on
  __device__ __forceinline__ int head(int kind) const { return p - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk); }
  __device__ __forceinline__ int left(int kind) const {
    const int n = (kind == 0 ? nq : kind == 1 ? nq + nk : all) - p;
    return n < rest ? n : rest;
  }
  // n passes on, all of one kind
  __device__ __forceinline__ void skip(int n) {
    rest -= n;
    p += n;
    if (p == all) {
      p = 0;
      ++group;
    }
  }
};

// What a warp loads, ahead of what it computes: a lane's rows of N arrays side by
// side (dy and x backward), into the stages of its ring.
template <class T, int N>
struct Loader {
  Walk w;
  const T* src[N];
  int64_t hop[N];  // from head to head
  int left;        // passes until the next kind of rows
  bool in;         // this lane has a column of a token
  __device__ __forceinline__ void begin(const Walk& at) {
    w = at;
    left = 0;
    in = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      src[i] = nullptr;
      hop[i] = 0;
    }
  }
  // The next pass, into the stage at `to`; nothing behind the last.  rows(kind, i): the i-th array's of a kind.
  template <bool INTER, class F>
  __device__ __forceinline__ void fetch(const RopeArgs& A, const Turn<INTER>& turn, int tokens, int sub, uint32_t to,
                                        const F& rows) {
    if (left == 0) {
      in = false;
      left = INT32_MAX;
      if (w.rest > 0) {
        const int kind = w.kind(), t = w.group * tokens + sub;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const RowsIn& r = rows(kind, i);
          src[i] = static_cast<const T*>(r.p) + t * r.token + w.head(kind) * r.head + turn.c;
          hop[i] = r.head;
        }
        in = turn.in && t < A.tokens;
        left = w.left(kind);
        w.skip(left);
      }
    }
    if (in)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        cp_async(to + i * 32 * Row<T>::kBytes, src[i]);
        cp_async(to + i * 32 * Row<T>::kBytes + Row<T>::kGroup, src[i] + turn.second);
      }
    cp_commit();
#pragma unroll
    for (int i = 0; i < N; ++i) src[i] += hop[i];
    --left;
  }
};

template <class T, int LANES, bool INTER, bool NORM, bool STORE>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int kTokens = 32 / LANES;
  constexpr uint32_t kStage = 32 * Row<T>::kBytes;  // of a warp
  constexpr int kStages = kRingBytes / (int)kStage;
  __shared__ __align__(16) uint8_t ring_all[kRopeThreads / 32 * kRingBytes];
  __shared__ __align__(16) float weights[2 * kWeights];
  const int lane = threadIdx.x & 31, sub = lane / LANES;
  const uint32_t ring = smem_u32(ring_all) + (threadIdx.x >> 5) * kRingBytes + lane * 16u;
  Turn<INTER> turn;
  turn.place(A, lane & (LANES - 1));
  if (!turn.in)  // columns past the row stay zeros
    for (uint32_t i = 0; i < kRingBytes; i += 512) st_shared4(ring + i, make_uint4(0, 0, 0, 0));
  const bool all_turned = A.rot == 8 * LANES;
  grid_begin();
  Walk at;
  at.begin(A, STORE ? 3 : 2, kTokens, (int)(blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5)));
  Loader<T, 1> ld;
  ld.begin(at);
  const auto fetch = [&](uint32_t to) {
    ld.fetch(A, turn, kTokens, sub, to,
             [&](int kind, int) -> const RowsIn& { return kind == 0 ? A.q : kind == 1 ? A.k : A.v; });
  };
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) fetch(ring + s * kStage);
  fill_weights<T>(A, weights);
  const float inv_dim = 1.0f / (float)A.dim;
  int pos = 0, t = 0;  // of the next group's token, until it is begun
  int64_t slot = -1;
  const auto look = [&](int group) {
    t = group * kTokens + sub;
    if (t >= A.tokens) return;
    pos = ld_plain(A.positions + t);
    if (STORE) slot = ld_plain(A.slots + t);
  };
  if (at.rest > 0) look(at.group);
  int token = 0;
  int64_t pool = -1;  // where the token's rows lie in the pools
  int begun = -1;     // the group whose angles are here
  uint32_t stage = 0;
#pragma unroll 1
  while (at.rest > 0) {
    if (begun != at.group) {
      begun = at.group;
      token = t;
      turn.at(A, pos);
      if (STORE) {
        const int64_t page = slot >> A.page_log2;
        const bool live = token < A.tokens && slot >= 0;
        if (live && page >= A.c.pages) raise_error(A.err, TP3D_EPAGES);
        pool = live && page < A.c.pages
                   ? page * A.c.page_stride + (slot & ((1 << A.page_log2) - 1)) * A.c.token_stride
                   : -1;
      }
      if (at.rest > at.all - at.p) look(at.group + 1);
    }
    // the passes of one kind
    const int kind = at.kind(), n = at.left(kind);
    bool out = turn.in && token < A.tokens;
    T* dst;
    int64_t hop;
    if (STORE && kind > 0) {
      dst = static_cast<T*>(kind == 1 ? A.c.k : A.c.v) + pool + at.head(kind) * A.c.head_stride + turn.c;
      hop = A.c.head_stride;
      out = out && pool >= 0;
    } else {
      const RowsOut& o = kind == 0 ? A.qo : A.ko;
      dst = static_cast<T*>(o.p) + token * o.token + at.head(kind) * o.head + turn.c;
      hop = o.head;
    }
    f32x2 a[4], b[4];
    {
      float w[8];
      columns_of(weights + (kind == 0 ? 0 : kWeights), turn.c, turn.second, w);
      turn.factors(w, false, a, b);
    }
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      cp_wait<kStages - 1>();
      Row<T> x;
      x.read(ring + stage);
      if (!STORE || kind < 2) {
        f32x2 y[4];
        x.get(y);
        if (NORM) {
          const f32x2 s = splat2(inverse_rms<LANES>(A.eps, y, inv_dim));
          turn.apply(y, a, b, all_turned);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], s);
        } else {
          turn.apply(y, a, b, all_turned);
        }
        x.set(y);
      }
      if (out) x.write(dst, turn.second);
      dst += hop;
      fetch(ring + stage);
      stage = (stage + kStage) & (kRingBytes - 1);
    }
    at.skip(n);
  }
}

// Backward: g = R(p)^T dy; with the norm dx = s (w g - x s^2 mean(w g x)) and the
// weights' gradients, the sums of g x s, kept in registers over a warp's tokens,
// joined warp by warp in shared memory and CTA by CTA in the workspace, in a
// fixed order; the last CTA to arrive adds the CTAs' parts.  Both sums of a row
// come out of five shuffles.  4096 tokens of 16 heads of 128 (101 MB): 25.4 us,
// 0.58 of the copy rate; without the weights' gradients 4 less, which are the
// parts' way through L2 (16384 tokens 71 and 67 us, 0.83).
template <class T, int LANES, bool INTER, bool NORM>
__global__ void __launch_bounds__(kBackThreads, 1) rope_back_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int kTokens = 32 / LANES, kWarps = kBackThreads / 32;
  constexpr uint32_t kHalf = 32 * Row<T>::kBytes, kStage = (NORM ? 2 : 1) * kHalf;  // dy, then x
  constexpr int kStages = kRingBytes / (int)kStage;
  extern __shared__ __align__(16) uint8_t back_smem[];
  float* const weights = reinterpret_cast<float*>(back_smem);
  uint8_t* const ring_all = back_smem + 2 * kWeights * sizeof(float);
  float* const sums = reinterpret_cast<float*>(ring_all);  // [warp][q or k][dim], when the ring is done with
  __shared__ int last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LANES;
  const uint32_t ring = smem_u32(ring_all) + warp * kRingBytes + lane * 16u;
  Turn<INTER> turn;
  turn.place(A, lane & (LANES - 1));
  if (!turn.in)
    for (uint32_t i = 0; i < kRingBytes; i += 512) st_shared4(ring + i, make_uint4(0, 0, 0, 0));
  const bool all_turned = A.rot == 8 * LANES;
  grid_begin();
  Walk at;  // neighbouring ranges to different CTAs: few fill the SMs evenly
  at.begin(A, 2, kTokens, warp * (int)gridDim.x + (int)blockIdx.x);
  Loader<T, NORM ? 2 : 1> ld;
  ld.begin(at);
  const auto fetch = [&](uint32_t to) {
    ld.fetch(A, turn, kTokens, sub, to, [&](int kind, int i) -> const RowsIn& {
      return i ? (kind == 0 ? A.q : A.k) : (kind == 0 ? A.dq : A.dk);
    });
  };
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) fetch(ring + s * kStage);
  fill_weights<T>(A, weights);
  const float inv_dim = 1.0f / (float)A.dim;
  f32x2 sq[4], sk[4], c[4], d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sq[i] = sk[i] = 0;
  int pos = 0, t = 0;
  const auto look = [&](int group) {
    t = group * kTokens + sub;
    if (t < A.tokens) pos = ld_plain(A.positions + t);
  };
  if (at.rest > 0) look(at.group);
  int token = 0, begun = -1;
  uint32_t stage = 0;
#pragma unroll 1
  while (at.rest > 0) {
    if (begun != at.group) {
      begun = at.group;
      token = t;
      turn.at(A, pos);
      const float ones[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
      turn.factors(ones, true, c, d);
      if (at.rest > at.all - at.p) look(at.group + 1);
    }
    const int kind = at.kind(), n = at.left(kind);
    const bool live = token < A.tokens;  // (what lies in the stage of a token past the last is no row)
    const RowsOut& o = kind == 0 ? A.qo : A.ko;
    T* dst = static_cast<T*>(o.p) + token * o.token + at.head(kind) * o.head + turn.c;
    f32x2 w[4], sum[4];
    {
      float v[8];
      columns_of(weights + (kind == 0 ? 0 : kWeights), turn.c, turn.second, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = pk2(v[2 * i], v[2 * i + 1]);
        sum[i] = 0;
      }
    }
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      cp_wait<kStages - 1>();
      Row<T> x;
      f32x2 g[4];
      x.read(ring + stage);
      x.get(g);
      turn.apply(g, c, d, all_turned);
      if (NORM) {
        f32x2 y[4];
        x.read(ring + stage + kHalf);
        x.get(y);
        // sum x^2 and sum w g x over the row together
        f32x2 q = mul2(y[0], y[0]), dot = 0, wg[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e) q = fma2(y[e], y[e], q);
          wg[e] = mul2(g[e], w[e]);
          dot = fma2(wg[e], y[e], dot);
        }
        float xx = sum_of(q), gx = sum_of(dot);
        row_sums<LANES>(xx, gx, lane);
        const float s = rsqrtf(fmaf(xx, inv_dim, A.eps));
        const f32x2 s2 = splat2(s), minus = splat2(-s * gx * inv_dim);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = mul2(y[e], s2);
          sum[e] = fma2(g[e], y[e], sum[e]);
          g[e] = mul2(fma2(y[e], minus, wg[e]), s2);
        }
      }
      x.set(g);
      if (turn.in && live) x.write(dst, turn.second);
      dst += o.head;
      fetch(ring + stage);
      stage = (stage + kStage) & (kRingBytes - 1);
    }
    if (live) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (kind == 0) sq[e] = add2(sq[e], sum[e]);
        else sk[e] = add2(sk[e], sum[e]);
      }
    }
    at.skip(n);
  }
  if (!A.parts) return;
  cp_wait<0>();
  __syncthreads();  // the ring is the sums' now
  const int width = 2 * A.dim;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    upk2(sq[i], v[0], v[1]);
    upk2(sk[i], v[2], v[3]);
    const int col = turn.c + (i < 2 ? 0 : turn.second) + 2 * (i & 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
      if (sub == 0 && turn.in) sums[warp * width + (e >> 1) * A.dim + col + (e & 1)] = v[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += kBackThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w * width + i];
    __stcg(A.parts + (size_t)blockIdx.x * width + i, s);
  }
  __syncthreads();
  if (threadIdx.x == 0) last = arrive_last(A.arrivals, gridDim.x);
  __syncthreads();
  if (!last) return;
  // four columns to a thread; group g of `groups` adds every groups-th part, then the groups are added
  const int quads = width / 4, fit = kBackThreads / quads, groups = fit < kWarps ? fit : kWarps;
  const int g = (int)threadIdx.x / quads, q = (int)threadIdx.x - g * quads;
  if (g < groups) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kFlight = 20;  // (all there are with heads of 128)
    for (int b0 = g; b0 < (int)gridDim.x; b0 += kFlight * groups) {
      float4 x[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (b0 + i * groups < (int)gridDim.x)
          x[i] = __ldcg(reinterpret_cast<const float4*>(A.parts + (size_t)(b0 + i * groups) * width) + q);
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (b0 + i * groups < (int)gridDim.x) s.x += x[i].x, s.y += x[i].y, s.z += x[i].z, s.w += x[i].w;
    }
    reinterpret_cast<float4*>(sums)[g * quads + q] = s;
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

// Cuts the passes (heads of groups of tokens) into equal ranges for `warps` warps; how many get one.
int64_t cut(RopeArgs& A, int lanes, int heads, int64_t warps) {
  const int64_t passes = ((int64_t)A.tokens + 32 / lanes - 1) / (32 / lanes) * heads;
  const int64_t range = (passes + warps - 1) / warps;
  A.range = (int32_t)range;
  return (passes + range - 1) / range;
}

template <class T, int LANES, bool STORE>
tp3d_status launch_rope_lanes(const tp3d_ctx* ctx, RopeArgs& A, int interleaved, cudaStream_t s) {
  const int per_cta = kRopeThreads / 32;
  const int64_t used = cut(A, LANES, A.heads + A.kv_heads * (STORE ? 2 : 1), (int64_t)ctx->num_sms * 3 * per_cta);
  const unsigned grid = (unsigned)((used + per_cta - 1) / per_cta);
  const auto kernel = interleaved ? (A.norm ? rope_kernel<T, LANES, true, true, STORE> : rope_kernel<T, LANES, true, false, STORE>)
                                  : (A.norm ? rope_kernel<T, LANES, false, true, STORE> : rope_kernel<T, LANES, false, false, STORE>);
  return launch_dependent(kernel, grid, kRopeThreads, 0, s, A);
}
template <class T, bool STORE>
tp3d_status launch_rope(const tp3d_ctx* ctx, RopeArgs& A, int interleaved, cudaStream_t s) {
  const int lanes = lanes_of(A.dim);
  if (lanes == 8) return launch_rope_lanes<T, 8, STORE>(ctx, A, interleaved, s);
  if (STORE || lanes == 16) return launch_rope_lanes<T, 16, STORE>(ctx, A, interleaved, s);  // (a cache's heads: 64 or 128)
  return launch_rope_lanes<T, STORE ? 16 : 32, STORE>(ctx, A, interleaved, s);
}

constexpr int kBackSmem = 2 * kWeights * (int)sizeof(float) + kBackThreads / 32 * kRingBytes;
static_assert(kBackThreads / 32 * 2 * kWeights * 4 <= kBackThreads / 32 * kRingBytes, "the sums fit into the ring");
template <class T, int LANES>
tp3d_status launch_back_lanes(tp3d_ctx* ctx, RopeArgs& A, int interleaved, cudaStream_t s) {
  const int64_t used = cut(A, LANES, A.heads + A.kv_heads, (int64_t)ctx->num_sms * (kBackThreads / 32));
  const unsigned grid = (unsigned)(used < ctx->num_sms ? used : ctx->num_sms);
  const auto kernel = interleaved ? (A.norm ? rope_back_kernel<T, LANES, true, true> : rope_back_kernel<T, LANES, true, false>)
                                  : (A.norm ? rope_back_kernel<T, LANES, false, true> : rope_back_kernel<T, LANES, false, false>);
  const unsigned bit = 1u << (8 + (LANES == 8 ? 0 : LANES == 16 ? 1 : 2) + (sizeof(T) == 4 ? 3 : 0) + (interleaved ? 6 : 0) +
                        (A.norm ? 12 : 0));
  if (!(ctx->paged_ready & bit)) {
    TP3D_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBackSmem));
    ctx->paged_ready |= bit;
  }
  return launch_dependent(kernel, grid, kBackThreads, kBackSmem, s, A);
}
template <class T>
tp3d_status launch_back(tp3d_ctx* ctx, RopeArgs& A, int interleaved, cudaStream_t s) {
  if (A.tokens == 0)
    return launch_dependent(rope_zero_kernel<T>, 1, 256, 0, s, static_cast<T*>(A.dqw), static_cast<T*>(A.dkw), A.dim);
  switch (lanes_of(A.dim)) {
    case 8: return launch_back_lanes<T, 8>(ctx, A, interleaved, s);
    case 16: return launch_back_lanes<T, 16>(ctx, A, interleaved, s);
    default: return launch_back_lanes<T, 32>(ctx, A, interleaved, s);
  }
}

tp3d_status check_counts(int64_t tokens, int heads, int kv_heads) {
  if (tokens < 0 || heads < 1 || kv_heads < 1) return TP3D_EINVAL;
  if (tokens > kPagedMaxTokens || heads > 65536 || kv_heads > 65536) return TP3D_EUNSUPPORTED;
  // (a warp's passes, 1 / 2432 of all on a device of 152 SMs, are counted in 32 bits)
  if (tokens * ((int64_t)heads + 2 * (int64_t)kv_heads) >> 40) return TP3D_EUNSUPPORTED;
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
