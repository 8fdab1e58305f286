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
__global__ void __launch_bounds__(kRowWarps * 32) paged_attn_row_kernel(const PagedAttn A) {
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
  if (r.n * A.group <= 64) return;
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

// ------------------------------------------------------------------ few rows
// Requests with at most kFewRows rows (new tokens x query heads) per key/value
// head: generation steps and short chunks.  Every row of a key/value head
// shares one read of its keys and values, so with few rows the cache's bytes
// bound the kernel: per key, 4 D bytes against 4 D rows FLOP, and HBM
// delivers a key in about the time the legacy tensor instructions
// (mma.sync, 16 rows x 8 keys x 16 columns) need a tenth of.
//
// Work is counted in tiles of KT keys of one (request, key/value head),
// request by request, head by head; the CTAs take equal contiguous ranges of
// that sequence, so one long request and many short ones balance alike and
// nothing about the lengths is needed on the host.  A CTA streams its tiles
// through a ring of shared-memory stages with 16-byte asynchronous copies
// (any page layout; keys past the request are zero-filled, so stale contents
// never reach a product).
//
// Four warps share a tile: with up to 16 rows each takes every fourth 16-key
// chunk, with up to 32 every second one of half the rows, with up to 64 all
// chunks of a quarter of them.  Each keeps its own running maximum (in base-2
// units; moved only when exceeded by more than 2^8, which leaves the
// probabilities far from overflow), row sums and D columns of O in registers.
//
// Where a range boundary cuts an item (request, head), each CTA leaves its
// part (maximum, sum, unnormalised O in fp32) in the workspace, and the CTA
// whose arrival completes the item's count adds the parts in key order.
constexpr int kFewThreads = 128;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 64;
constexpr int kFewStages = 3;
constexpr int kFewPerSm = 2;
constexpr uint32_t kFewStageBytes = 32768;  // a tile's keys, then its values
constexpr float kMoveLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
TP3D_HD constexpr int few_tile_keys() { return (int)kFewStageBytes / (4 * D); }

struct FewShared {
  float m[kFewWarps][16], l[kFewWarps][16];
  long long scan[kFewWarps];
  long long before;  // units before request `b0` (the CTA's first)
  int b0;
  int last;
  int poisoned;
  int poison[128];  // per column: the first key with a non-finite value in a partly masked tile
};

template <int D>
constexpr size_t few_smem() { return (size_t)kFewStages * kFewStageBytes + sizeof(FewShared) + 128; }

TP3D_HD constexpr size_t few_part_floats(int d) { return (size_t)kFewRows * (d + 2); }

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c (16 x 8, fp32) += a (16 x 16, bf16) b (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The equal contiguous ranges of `units` units over `n` CTAs, and the CTA that unit u belongs to.
struct Ranges {
  int64_t base, rem;
  __device__ Ranges(int64_t units, int64_t n) : base(units / n), rem(units % n) {}
  __device__ int64_t begin(int64_t c) const { return c * base + (c < rem ? c : rem); }
  __device__ int64_t owner(int64_t u) const {
    const int64_t big = rem * (base + 1);
    return u < big ? u / (base + 1) : rem + (u - big) / base;
  }
};

// A position in the sequence of tiles: tile `tile` of `tiles` of (request b, head h).
struct FewCursor {
  int b, h, tile, tiles, n, kv;
  int64_t q0;
};

// tiles of request b (0: not this kernel's)
template <int D>
__device__ __forceinline__ int few_tiles(const PagedAttn& A, int b, PagedRequest* r, bool alone) {
  *r = paged_request(A, b);
  const int64_t rows = (int64_t)r->n * A.group;
  if (rows == 0) return 0;
  if (rows > kFewRows) {
    if (alone) raise_error(A.err, TP3D_EPAGES);
    return 0;
  }
  constexpr int KT = few_tile_keys<D>();
  return r->kv > 0 ? (r->kv - 1) / KT + 1 : 1;  // a request without keys still has rows to write
}

template <int D>
__device__ __forceinline__ void few_enter(const PagedAttn& A, FewCursor& c, bool alone) {
  PagedRequest r;
  c.tiles = few_tiles<D>(A, c.b, &r, alone);
  c.n = r.n;
  c.kv = r.kv;
  c.q0 = r.q0;
}
template <int D>
__device__ __forceinline__ void few_advance(const PagedAttn& A, FewCursor& c, bool alone) {
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.h < A.c.kv_heads) return;
  c.h = 0;
  do {
    ++c.b;
    few_enter<D>(A, c, alone);
  } while (c.tiles == 0);
}

// `alone`: no other kernel of the call takes the requests with more rows
template <int D>
__global__ void __launch_bounds__(kFewThreads, kFewPerSm)
    paged_attn_few_kernel(const PagedAttn A, bool alone, float* __restrict__ parts, unsigned* __restrict__ counters) {
  constexpr int KT = few_tile_keys<D>(), NG = KT / 16, RV = D / 8, NT = D / 8;  // RV: 16-byte vectors of a row
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const tiles_ptr = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  const uint32_t stages = smem_u32(tiles_ptr);
  FewShared& sh = *reinterpret_cast<FewShared*>(tiles_ptr + kFewStages * kFewStageBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- this CTA's range of the tile sequence
  int64_t units = 0, u0 = 0, u1 = 0;
  {
    // sums of the tiles over the requests, kFewThreads at a time; the second
    // pass finds the request of the range's first tile
    long long carry = 0;
    auto chunk = [&](int base, long long& mine, int& tiles) {
      PagedRequest r;
      const int b = base + tid;
      tiles = b < A.requests ? few_tiles<D>(A, b, &r, alone) : 0;
      long long x = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) sh.scan[warp] = x;
      __syncthreads();
      mine = carry + x - tiles;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        if (w < warp) mine += sh.scan[w];
        carry += sh.scan[w];
      }
    };
    long long mine = 0;
    int tiles = 0;
    for (int base = 0; base < A.requests; base += kFewThreads) chunk(base, mine, tiles);
    units = carry * A.c.kv_heads;
    const Ranges R(units, gridDim.x);
    u0 = R.begin(blockIdx.x);
    u1 = R.begin(blockIdx.x + 1);
    if (u0 >= u1) return;
    const bool one = A.requests <= kFewThreads;
    carry = 0;
    for (int base = 0; base < A.requests; base += kFewThreads) {
      if (!one) chunk(base, mine, tiles);
      const long long at = mine * A.c.kv_heads;
      if (tiles > 0 && at <= u0 && u0 < at + (long long)tiles * A.c.kv_heads) {
        sh.b0 = base + tid;
        sh.before = at;
      }
      if (one || carry * A.c.kv_heads > u0) break;
    }
    for (int i = tid; i < 128; i += kFewThreads) sh.poison[i] = INT32_MAX;
    if (tid == 0) sh.poisoned = 0;
    __syncthreads();
  }
  const Ranges ranges(units, gridDim.x);
  FewCursor c;
  c.b = sh.b0;
  few_enter<D>(A, c, alone);
  {
    const int64_t off = u0 - sh.before;
    c.h = (int)(off / c.tiles);
    c.tile = (int)(off - (int64_t)c.h * c.tiles);
  }

  // ---- loads: thread -> vector (tid % RV) of rows tid / RV + i * (kFewThreads / RV)
  const bf16* const kpool = static_cast<const bf16*>(A.c.k);
  const bf16* const vpool = static_cast<const bf16*>(A.c.v);
  FewCursor ld = c;
  int64_t lu = u0;  // the unit that ld stands at
  int32_t ld_page = 0;  // the page of 16-key group (lane % NG) of that tile; -1: none
  auto fetch_pages = [&]() {
    const int64_t key = (int64_t)ld.tile * KT + (lane & (NG - 1)) * 16;
    ld_page = -1;
    if (key < ld.kv) {
      ld_page = __ldg(A.table + (int64_t)ld.b * A.width + (key >> A.page_log2));
      if (ld_page < 0 || ld_page >= A.c.pages) {
        raise_error(A.err, TP3D_EPAGES);
        ld_page = -1;
      }
    }
  };
  auto load = [&](int stage) {
    constexpr int RS = kFewThreads / RV;  // rows per step: 8 or 16
    const int v = tid & (RV - 1), r0 = tid / RV;
    const uint32_t base = stages + (uint32_t)stage * kFewStageBytes;
#pragma unroll
    for (int i = 0; i < KT / RS; ++i) {
      const int r = r0 + i * RS;
      const int32_t page = __shfl_sync(0xffffffffu, ld_page, (i * RS) >> 4);  // 16 rows share a page
      const int64_t key = (int64_t)ld.tile * KT + r;
      const bool in = page >= 0 && key < ld.kv;
      const int64_t at = in ? (int64_t)page * A.c.page_stride + (key & (A.c.page - 1)) * A.c.token_stride +
                                  ld.h * A.c.head_stride + v * 8
                            : 0;
      // vector v of row r at v ^ (r mod 8): the eight rows of an 8 x 8 block fall in different banks
      const uint32_t dst = base + (uint32_t)(r * RV + (v ^ (r & 7))) * 16u;
      cp_async16_zfill(dst, kpool + at, in);
      cp_async16_zfill(dst + kFewStageBytes / 2, vpool + at, in);
    }
  };
  fetch_pages();
  for (int s = 0; s < kFewStages - 1; ++s) {
    if (lu < u1) {
      load(s);
      if (++lu < u1) {
        few_advance<D>(A, ld, alone);
        fetch_pages();
      }
    }
    cp_commit();
  }

  const float sl2 = A.scale * kLog2e;
  uint32_t qf[D / 16][4];
  float o[NT][4], m[2], l[2];
  int lim[2];  // the last key that this thread's two rows see
  int WM = 1, stage = 0;
  bool begin = true;
  for (int64_t u = u0; u < u1; ++u) {
    cp_wait<kFewStages - 2>();
    __syncthreads();  // the tile of unit u is in; everybody is done with unit u - 1's
    {
      const int s = stage == 0 ? kFewStages - 1 : stage - 1;
      if (lu < u1) {
        load(s);
        if (++lu < u1) {
          few_advance<D>(A, ld, alone);
          fetch_pages();
        }
      }
      cp_commit();
    }
    const int rows = c.n * A.group;
    if (begin) {
      WM = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
      begin = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = (warp & (WM - 1)) * 16 + (lane >> 2) + 8 * e;
        const bool in = r < rows;
        const int tok = in ? r / A.group : 0, g = in ? r - tok * A.group : 0;
        lim[e] = in ? c.kv - c.n + tok : c.kv - 1;
        const bf16* src = A.q + (c.q0 + tok) * A.q_token + (int64_t)(c.h * A.group + g) * A.q_head + (lane & 3) * 2;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][e] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + k * 16)) : 0u;
          qf[k][2 + e] = in ? __ldg(reinterpret_cast<const uint32_t*>(src + k * 16 + 8)) : 0u;
        }
        m[e] = -INFINITY;
        l[e] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    }
    const int WK = kFewWarps / WM;
    const uint32_t sk = stages + (uint32_t)stage * kFewStageBytes, sv = sk + kFewStageBytes / 2;
    // keys of this tile that some row does not see: past kv - n (kv when n = 1)
    const bool partial = (int64_t)(c.tile + 1) * KT - 1 > (int64_t)c.kv - c.n;
    for (int kc = warp / WM; kc < NG; kc += WK) {
      const int key0 = c.tile * KT + kc * 16;
      if (key0 >= c.kv) break;
      // S = Q K^T for 16 keys: two 8-key tiles, two partial sums each
      float s[2][2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][y][e] = 0.0f;
      {
        const int row = kc * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int vec = 2 * k + ((lane >> 3) & 1);
          uint32_t kb[4];
          ldmatrix4(kb, sk + (uint32_t)(row * RV + (vec ^ (row & 7))) * 16u);
          mma16816(s[0][k & 1], qf[k], kb[0], kb[1]);
          mma16816(s[1][k & 1], qf[k], kb[2], kb[3]);
        }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[x][0][e] + s[x][1][e];
          if (partial && key0 + x * 8 + (lane & 3) * 2 + (e & 1) > lim[e >> 1]) v = -INFINITY;
          s[x][0][e] = v;
          mx[e >> 1] = fmaxf(mx[e >> 1], v);
        }
      bool move = false;
      float mt[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        mt[e] = mx[e] * sl2;
        move |= mt[e] > m[e] + kMoveLog2;
      }
      if (__any_sync(0xffffffffu, move)) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool mv = mt[e] > m[e] + kMoveLog2;
          f[e] = mv ? ex2_approx(m[e] - mt[e]) : 1.0f;
          if (mv) m[e] = mt[e];
          l[e] *= f[e];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= f[e >> 1];
      }
      const float mb[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = ex2_approx(fmaf(s[x][0][e], sl2, -mb[e >> 1]));
          s[x][0][e] = p;
          l[e >> 1] += p;
        }
      // O += P V.  V is bf16, so P enters as two bf16 terms, P = hi + lo up to
      // 2^-17 P: rounded to one, its error alone would be as large as the
      // output's own rounding.  The second product costs no time here.
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = s[i >> 1][0][2 * (i & 1)], y = s[i >> 1][0][2 * (i & 1) + 1];
        ph[i] = pack_bf16(x, y);
        pl[i] = pack_bf16(x - __uint_as_float(ph[i] << 16), y - __uint_as_float(ph[i] & 0xffff0000u));
      }
      const int row = kc * 16 + (lane & 15);
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        const int vec = j + (lane >> 4);
        uint32_t vb[4];
        ldmatrix4_trans(vb, sv + (uint32_t)(row * RV + (vec ^ (row & 7))) * 16u);
        if (partial && c.n > 1) {
          // A probability of 0 does not silence a value that is not finite:
          // such a value becomes 0 here, and rows that see its key get NaN in
          // its column at the end.
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (((vb[x] >> (16 * e)) & 0x7f80u) == 0x7f80u) {
                vb[x] &= e ? 0x0000ffffu : 0xffff0000u;
                atomicMin(&sh.poison[(j + (x >> 1)) * 8 + (lane >> 2)],
                          key0 + (x & 1) * 8 + (lane & 3) * 2 + e);
                sh.poisoned = 1;
              }
        }
        mma16816(o[j], ph, vb[0], vb[1]);
        mma16816(o[j + 1], ph, vb[2], vb[3]);
        mma16816(o[j], pl, vb[0], vb[1]);
        mma16816(o[j + 1], pl, vb[2], vb[3]);
      }
    }

    // ---- the item's last tile, or this CTA's: join the warps and write
    if (c.tile + 1 == c.tiles || u + 1 == u1) {
      const int64_t item0 = u - c.tile;  // the item's first unit
      const bool whole = item0 >= u0 && c.tile + 1 == c.tiles;
      __syncthreads();  // every warp is done with the tile: its stage takes the parts
      float* const so = reinterpret_cast<float*>(tiles_ptr + (size_t)stage * kFewStageBytes);  // [warp][16][D]
      const auto swz = [](int r, int col) { return r * D + (col ^ ((r & 3) << 3)); };
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        const int r = (lane >> 2) + 8 * e;
        if ((lane & 3) == 0) {
          sh.m[warp][r] = m[e];
          sh.l[warp][r] = l[e];
        }
        const bool hurt = sh.poisoned != 0;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int col = j * 8 + (lane & 3) * 2;
          float2 v = make_float2(o[j][2 * e], o[j][2 * e + 1]);
          if (hurt) {
            if (sh.poison[col] <= lim[e]) v.x = __int_as_float(0x7fffffff);
            if (sh.poison[col + 1] <= lim[e]) v.y = __int_as_float(0x7fffffff);
          }
          *reinterpret_cast<float2*>(so + warp * 16 * D + swz(r, col)) = v;
        }
      }
      __syncthreads();
      const int c0 = whole ? 0 : (int)ranges.owner(item0);
      const int pieces = whole ? 1 : (int)ranges.owner(item0 + c.tiles - 1) - c0 + 1;
      const size_t pf = few_part_floats(D);
      // a part that begins its item is its CTA's last piece, slot 1; one that continues it the first, slot 0
      float* const part = parts + ((size_t)blockIdx.x * 2 + (item0 >= u0 ? 1 : 0)) * pf;
      const auto finish = [&](int r, int col, float4 v, float top, float sum) {
        const int tok = r / A.group;
        const int64_t t = c.q0 + tok;
        const int head = c.h * A.group + (r - tok * A.group);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        *reinterpret_cast<uint2*>(A.o + t * A.o_token + (int64_t)head * A.o_head + col) =
            make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
        if (A.lse && col == 0)
          A.lse[t * (int64_t)(A.group * A.c.kv_heads) + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
      };
      const int elems = rows * (D / 4);
      for (int i = tid; i < elems; i += kFewThreads) {
        const int r = i / (D / 4), col = (i - r * (D / 4)) * 4, rt = r >> 4, rr = r & 15;
        float top = -INFINITY, sum = 0.0f;
        for (int w = rt; w < kFewWarps; w += WM) top = fmaxf(top, sh.m[w][rr]);
        const float tb = top == -INFINITY ? 0.0f : top;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = rt; w < kFewWarps; w += WM) {
          const float f = ex2_approx(sh.m[w][rr] - tb);
          const float4 v = *reinterpret_cast<const float4*>(so + w * 16 * D + swz(rr, col));
          sum += f * sh.l[w][rr];
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        if (whole) {
          finish(r, col, acc, tb, sum);
        } else {
          __stcg(reinterpret_cast<float4*>(part + (size_t)r * D + col), acc);
          if (col == 0) {
            __stcg(part + kFewRows * D + r, top);
            __stcg(part + kFewRows * (D + 1) + r, sum);
          }
        }
      }
      if (!whole) {
        __threadfence();
        __syncthreads();
        // the count returns to zero with the item's last arrival
        if (tid == 0) sh.last = atomicInc(counters + c0, (unsigned)pieces - 1) == (unsigned)pieces - 1;
        __syncthreads();
        if (sh.last) {
          __threadfence();
          for (int i = tid; i < elems; i += kFewThreads) {
            const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
            const auto at = [&](int p) { return parts + ((size_t)(c0 + p) * 2 + (p == 0 ? 1 : 0)) * pf; };
            float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
            for (int p = 0; p < pieces; ++p) top = fmaxf(top, __ldcg(at(p) + kFewRows * D + r));
            const float tb = top == -INFINITY ? 0.0f : top;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int p = 0; p < pieces; ++p) {
              const float f = ex2_approx(__ldcg(at(p) + kFewRows * D + r) - tb);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(at(p) + (size_t)r * D + col));
              sum += f * __ldcg(at(p) + kFewRows * (D + 1) + r);
              acc.x += f * v.x;
              acc.y += f * v.y;
              acc.z += f * v.z;
              acc.w += f * v.w;
            }
            finish(r, col, acc, tb, sum);
          }
        }
      }
      begin = true;
      if (sh.poisoned) {
        __syncthreads();
        for (int i = tid; i < 128; i += kFewThreads) sh.poison[i] = INT32_MAX;
        if (tid == 0) sh.poisoned = 0;
      }
    }
    if (u + 1 < u1) few_advance<D>(A, c, alone);
    stage = stage == kFewStages - 1 ? 0 : stage + 1;
  }
  cp_wait<0>();
}

}  // namespace

size_t paged_attn_workspace(const tp3d_ctx* ctx, int d) {
  return (size_t)ctx->num_sms * kFewPerSm * 2 * few_part_floats(d) * sizeof(float);
}

template <int D>
static tp3d_status launch_few(tp3d_ctx* ctx, const PagedAttn& A, bool alone, void* workspace, cudaStream_t s) {
  TP3D_CUDA_TRY(cudaFuncSetAttribute(paged_attn_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)few_smem<D>()));
  paged_attn_few_kernel<D><<<ctx->num_sms * kFewPerSm, kFewThreads, few_smem<D>(), s>>>(
      A, alone, static_cast<float*>(workspace), ctx->d_paged);
  return cudaGetLastError() == cudaSuccess ? TP3D_OK : TP3D_ECUDA;
}

tp3d_status launch_paged_attn(tp3d_ctx* ctx, const PagedAttn& A, int max_new, void* workspace, cudaStream_t s) {
  if (ctx->num_sms * kFewPerSm > kPagedCounters) return TP3D_EUNSUPPORTED;
  const int heads = A.group * A.c.kv_heads;
  const int64_t most = (max_new > 0 && max_new < A.tokens ? max_new : A.tokens) * A.group;
  const bool alone = most <= kFewRows;
  TP3D_TRY(A.c.head_dim == 128 ? launch_few<128>(ctx, A, alone, workspace, s)
                               : launch_few<64>(ctx, A, alone, workspace, s));
  if (alone) return TP3D_OK;
  if (heads > 65535) return TP3D_EUNSUPPORTED;
  const dim3 grid((unsigned)A.tokens, (unsigned)heads);
  if (A.c.head_dim == 128)
    paged_attn_row_kernel<128><<<grid, kRowWarps * 32, 0, s>>>(A);
  else
    paged_attn_row_kernel<64><<<grid, kRowWarps * 32, 0, s>>>(A);
  return cudaGetLastError() == cudaSuccess ? TP3D_OK : TP3D_ECUDA;
}

}  // namespace tp3d
