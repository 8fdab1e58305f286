// paged_attn.cu - attention of new tokens over the paged key/value cache.
//
// Row (t, i) of request b (new token j = t - q_start_b, query head i) sees
// the keys k = 0 .. kv_b - n_b + j:
//   s_k = scale q . k_k,  m = max s_k,  l = sum exp(s_k - m),
//   O = sum exp(s_k - m) v_k / l,  lse = m + log l,
// in one pass over the keys with a running m, l and O.  With a window of w
// keys and f first ones that stay visible, the row at position p sees of these
// only k > p - w and k < f (WIN in the kernels).
#include <cudaTypedefs.h>
#include <math.h>

#include "attn_tile.cuh"
#include "paged.cuh"

namespace tp3d {

namespace {

// ------------------------------------------------------------------ few rows
// Requests with few rows (new tokens x query heads; see kRows) per key/value
// head: generation steps and short chunks.  Every row of a key/value head
// shares one read of its keys and values, so the cache's bytes bound the
// kernel: per key, 4 D bytes against 4 D rows FLOP, which the legacy tensor
// instructions (mma.sync, 16 rows x 8 keys x 16 columns) do several times
// faster than HBM delivers them.
//
// Work is counted in tiles of 64 or 128 keys of one item (request, key/value
// head, 16 rows), request by request, head by head; the CTAs take equal
// contiguous ranges of that sequence, so one long request and many short ones
// balance alike and nothing about the lengths is needed on the host.  Each of a
// CTA's warps takes 16 keys of every tile - one page holds them all - through a ring of
// its own, with 16-byte asynchronous copies and no barrier between the warps:
// a warp refills a stage as soon as it has read it, which keeps one of two
// stages in flight, 64 KiB an SM; with three the same bytes come more slowly (32
// requests of up to 16384 keys 190 us against 182, one of 131071 91.9 against
// 87.5, short calls the same) (keys past the request are zero-filled, so stale contents
// never reach a product).  Each keeps its own running maximum (in base-2
// units; moved only when exceeded by more than 2^8, which leaves the
// probabilities far from overflow), row sums and O in registers; they are
// joined at the end of an item (request, head).
//
// Where a range boundary cuts an item, each CTA leaves its part (maximum, sum,
// unnormalised O in fp32) in the workspace, and the CTA whose arrival
// completes the item's count adds the parts in key order.
//
// A short call spends most of its time on instructions fetched for the first
// time, so what runs once is written as rolled loops, and loads are issued in
// one place.
//
// Measured, of a stream of calls: 32 requests of up to 16384 keys, 32 heads on 8,
// pages of 64 with the heads outside (1185 MB): 182 us, 6.5 TB/s, 0.97 of the
// copy rate.  32 of up to 4096, 16 heads, pages of 16 with the tokens outside
// (539 MB): 87 us, 0.93: rows of 256 bytes 4 KiB apart.  DRAM reads are the
// cache's bytes and no more.  A call of one tile: 4.7 us, of which 0.8 is the
// launch, 0.9 the lengths, 2 the table's page and then its keys; a cut item adds
// 3 for its parts' way through L2.
//
// W warps a CTA, 8 / W CTAs an SM.  Four: one CTA's end of an item falls
// together with another's loads.  Eight: fewer parts to an item and fewer steps
// to a part, where the items are too few to give every SM its own.  4 | 8
// warps: 16 items of 1024 keys 9.7 | 8.4 us, 16 of 3000 12.9 | 10.6, 64 of 1024
// 11.5 | 9.8, 8 of 131072 88.2 | 87.6; 128 items of 1024 13.3 | 15.0, 96 of 2000
// 15.5 | 20.0, 512 of 4096 96 | 107.
template <int W>
struct FewShape {
  static constexpr int kThreads = 32 * W;
  static constexpr int kKeys = 16 * W;  // of a tile
  static constexpr int kPerSm = 8 / W;
  // tiles of a CTA's range, where there is little work (16 items of 1024 keys, four warps: 9.7 us; with 2 10.3, with
  // 6 12.6; eight warps: 8.4 us; with 1 9.1, with 3 10.2)
  static constexpr int kMinTiles = 16 / W;
  // Rows of a request that this kernel takes, in blocks of 16 (items of their
  // own, side by side, so that a block finds the others' keys in L2).  Here | in
  // the kernel for many rows, eight warps: 4 requests of up to 2000 keys, 4
  // heads, 24 rows 12.0 | 21.4 us, 48 rows 13.1 | 22.1, 64 rows 18.0 | 22.2; one of
  // 65536, 4 heads, 24 rows 41.4 | 59.2, 48 rows 60.5 | 62.2, 64 rows 73.0 | 62.5.
  // Four warps: 64 of up to 500, 8 heads of 64, 16 rows 17.8 | 30.5.  (There more
  // rows would gain too, which the limit does not use: 20 rows 18.3 | 27.8; 32 of
  // up to 4000, 8 heads, 32 rows 90.9 | 100.2; 16 of up to 2000, 16 heads, 30
  // rows 41.2 | 53.1.)
  static constexpr int kRows = W == 8 ? 48 : 16;
  // With a window, where the host knows how many keys a row sees: blocks beside one another in either shape, and two of
  // them pay with four warps too, for heads of 64 at any window, for heads of 128 at short ones.  Here | there, 32
  // rows: 128 items, heads of 64, 8.4 | 13.9 us (window 128), 25.7 | 32.3 (1167), 61.8 | 72.7 (4096); 512 items 25.1 |
  // 33.4, 78.6 | 93.3, 223 | 238; heads of 128, 128 items 10.8 | 15.2, 34.1 | 38.0, 83.2 | 84.7, 512 items 35.4 | 36.9, 110
  // | 107, 330 | 275.  48 rows lose but for very short windows: 128 items of 64 13.9 | 14.1, 22.9 | 20.0 (512).
  // With heads of 128 the limit does not win everywhere.  Over 80 to 512 items, 20 to 32 rows and windows of 128 to
  // 1280, lengths alike and not, the time here is 0.61 to 1.16 of that there, 0.87 in the mean, above 1.03 at 79 of
  // 1096 points: where the ends of tiles and ranges fall badly, 112 to 144 items with windows of 384 to 704 0.65 to 1.16 (0.97 in the mean; 128
  // items, 32 rows, window 512: 25.2 | 22.6, 448 with unequal lengths 0.86), 256 of 512 37.4 | 36.2, 384 and 512 items
  // of 128 to 256 0.86 to 1.12.  No limit on items and window tells these from their neighbours.
  static constexpr int kRowsWindow = 32, kKeysWindow = 1280;
  // The end of an item counts as so many tiles in the ranges, about what it costs.  With it | without, four warps:
  // 32 requests of up to 4096 keys, 16 heads 85 | 94 us (one box); 100 of 700 41.8 | 60.9; 200 of 2000, 8 heads 127 | 145 (1:
  // 131, 3: 128).  With eight an item has several CTAs.
  static constexpr int kEnd = W == 8 ? 0 : 2;
  static constexpr int kSnap = 8 / W;  // a range boundary this near an item's edge moves there: parts cost more
};
constexpr int kFewRows = 16;  // of an item: one mma.sync tile
constexpr int kFewStages = 2;  // of a warp's ring
constexpr int kJoinOnce = 16;    // parts of an item joined in one step (8 heads of 64, 60000 keys: 13.2 us; all 152 at once 30.1)
constexpr int kFewSlots = 4;     // parts that a CTA has room for in the workspace
constexpr float kMoveLog2 = 8.0f;

template <int W>
struct FewShared {
  float m[W][16], l[W][16];
  long long scan[W];
  int before;  // units before request `b0` (the CTA's first)
  int b0;
  int last;
  int poisoned;
  // per column: the first key with a non-finite value that some row does not see; with a window the rows of the
  // block that see such a key, a bit each
  int poison[128];
};

TP3D_HD constexpr uint32_t few_stage_bytes(int d) { return 16u * 4u * (uint32_t)d; }  // 16 keys, then 16 values
template <int W>
constexpr size_t few_smem(int d) {
  return (size_t)W * kFewStages * few_stage_bytes(d) + sizeof(FewShared<W>) + 128;
}
TP3D_HD constexpr size_t few_part_floats(int d) { return (size_t)kFewRows * (d + 2); }

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
// Adds 0 times each of the eight bf16 of x to acc (two sums): they stay zeros
// while the values are finite and become NaN, for good, with one that is not.
__device__ __forceinline__ void watch_finite(__nv_bfloat162& acc, const uint4& x) {
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __hfma2(h[i], zero, acc);
}
__device__ __forceinline__ bool saw_not_finite(const __nv_bfloat162& acc) {
  return (*reinterpret_cast<const uint32_t*>(&acc) & 0x7fff7fffu) != 0;
}
// Sets the non-finite ones of the eight bf16 of x to zero; note(i) for each.
template <class Note>
__device__ __forceinline__ uint4 make_finite(const uint4& x, const Note& note) {
  uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const uint32_t mask = 0x7f80u << (16 * (i & 1));
    uint32_t word = e[0];
#pragma unroll
    for (int q = 1; q < 4; ++q) word = (i >> 1) == q ? e[q] : word;
    if ((word & mask) != mask) continue;
    word &= i & 1 ? 0x0000ffffu : 0xffff0000u;
#pragma unroll
    for (int q = 0; q < 4; ++q) e[q] = (i >> 1) == q ? word : e[q];
    note(i);
  }
  return make_uint4(e[0], e[1], e[2], e[3]);
}

// What a row's unnormalised O is multiplied by.  A sum of 0 is a row without
// keys (`last` < 0, the last key it sees), whose O is 0, or one that sees
// nothing but scores of -infinity: 0 / 0.
__device__ __forceinline__ float normaliser(float sum, int last) {
  return sum != 0.0f ? 1.0f / sum : last < 0 ? 0.0f : __int_as_float(0x7fffffff);
}

// The CTAs' equal contiguous shares of a sequence of units, and the CTA whose
// share unit u falls in.  In 32 bits: a call of 2^31 tiles or more raises
// TP3D_EPAGES instead (64-bit division costs a short call a microsecond).
struct Ranges {
  unsigned base, rem;
  __device__ Ranges(unsigned units, unsigned n) : base(units / n), rem(units % n) {}
  __device__ int begin(unsigned c) const { return (int)(c * base + (c < rem ? c : rem)); }
  __device__ int owner(unsigned u) const {
    const unsigned big = rem * (base + 1);
    return (int)(u < big ? u / (base + 1) : rem + (u - big) / base);
  }
};

// With a window the keys of a request that none of its new rows sees lie
// between the first keys and the first row's window: [first, low).  Tiles that
// hold nothing else are left out of the sequence: of a request's tiles the first
// `lead` are its first ones, and `gap` are missing behind them.
struct Gap {
  int lead = 0, gap = 0;
  __device__ void set(int first_tiles, int low_tile) {
    lead = first_tiles < low_tile ? first_tiles : low_tile;
    gap = low_tile - lead;
  }
  // a tile's number among all
  __device__ int tile(int j) const { return j >= lead ? j + gap : j; }
  // the position of the first tile there is from tile t on
  __device__ int at(int t) const { return t < lead ? t : t - gap > lead ? t - gap : lead; }
};
// the first key in the window of the row at position p
__device__ __forceinline__ int window_begin(int p, int window) { return p >= window ? p - window + 1 : 0; }

// A position in a CTA's range: tile `tile`, below `end`, of the `tiles` of
// (request b, head h, rows from row0), whose first is unit `at`.
template <int W, bool WIN>
struct FewCursor {
  using Shape = FewShape<W>;
  static constexpr bool kBlocks = WIN || Shape::kRows > 16;  // a request may have several
  Gap gap;
  int low;  // the first key of the first row's window
  int b, h, row0, tile, end, tiles, n, kv, at, u1;  // u1: the range's end (before it is moved)
  int64_t q0;
  // takes request b; tiles = 0 where it is not this kernel's
  __device__ void take(const PagedAttn& A, bool alone) {
    const PagedRequest r = paged_request(A, b);
    n = r.n;
    kv = r.kv;
    q0 = r.q0;
    const int64_t rows = (int64_t)n * A.group;
    tiles = kv > 0 ? (kv - 1) / Shape::kKeys + 1 : 1;  // a request without keys still has rows to write
    if (WIN) {
      low = window_begin(kv - n, A.window);
      const int first = A.sinks < kv ? A.sinks : kv;
      gap.set((first + Shape::kKeys - 1) / Shape::kKeys, low / Shape::kKeys);
      tiles -= gap.gap;
    }
    if (rows == 0 || rows > A.few_rows) {
      tiles = 0;
      if (alone && rows) raise_error(A.err, TP3D_EPAGES);
    }
  }
  // the first key of the item's tile t
  __device__ int key(int t) const { return (WIN ? gap.tile(t) : t) * Shape::kKeys; }
  // keys [k, k + 16) are seen by no row
  __device__ bool unseen(const PagedAttn& A, int k) const { return WIN && k >= A.sinks && k + 16 <= low; }
  // an item's length in the sequence
  __device__ int span() const { return tiles + Shape::kEnd; }
  // blocks of 16 rows (of a request that is this kernel's)
  __device__ int blocks(const PagedAttn& A) const { return kBlocks ? (n * A.group + 15) / 16 : 1; }
  // where a boundary `off` tiles into an item comes to lie
  __device__ int snap(int off) const {
    const int rest = tiles - off;
    return (off < rest ? off : rest) > Shape::kSnap ? off : off <= rest ? 0 : tiles;
  }
  // the range's share of this item: false when it ends before it
  __device__ bool share() {
    const int left = u1 - at;
    end = left >= tiles ? tiles : left > 0 ? snap(left) : 0;
    return end > tile;
  }
  __device__ bool next_item(const PagedAttn& A, bool alone) {
    tile = 0;
    at += span();
    if (at >= u1) return false;
    row0 += 16;
    if (kBlocks && row0 < n * A.group) return share();
    row0 = 0;
    if (++h == A.c.kv_heads) {
      h = 0;
      do {
        ++b;
        take(A, alone);
      } while (tiles == 0);
    }
    return share();
  }
  __device__ bool advance(const PagedAttn& A, bool alone) {
    if (++tile < end) return true;
    return end == tiles && next_item(A, alone);
  }
};

// A call's kernel for few rows begins beside its kernel for many, so its own
// wait (for the end of that one) comes last; what it reads, kernels before
// that one have written.  The other kernel's first CTA says in a word that its
// wait, and so all of those writes, is behind it; each CTA here acquires the
// word, or, if it does not find it, waits like any kernel.  The first CTA
// clears it for the next call at its own end, when the other kernel has ended
// and whoever looks later need not wait.  Waiting in every CTA instead: the
// mixed batch of 16 requests 101.9 us against 95.7.
__device__ __forceinline__ void say_waited(unsigned* word) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(word), "r"(1u) : "memory");
}
__device__ __forceinline__ void see_waited(unsigned* word) {
  unsigned seen;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(word) : "memory");
  if (!seen) grid_wait();
}

// `alone`: no other kernel of the call takes the requests with more rows
template <int D, int W, bool WIN>
__global__ void __launch_bounds__(FewShape<W>::kThreads, FewShape<W>::kPerSm)
    paged_attn_few_kernel(const PagedAttn A, bool alone, float* __restrict__ parts, unsigned* __restrict__ counters,
                          unsigned* waited) {
  using Shape = FewShape<W>;
  constexpr int kThreads = Shape::kThreads, kKeys = Shape::kKeys;
  constexpr int RV = D / 8, NT = D / 8;  // 16-byte vectors of a row, 8-column tiles of O
  constexpr uint32_t kStage = few_stage_bytes(D);
  constexpr int kNoPoison = WIN ? 0 : INT32_MAX;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const ring_ptr = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  FewShared<W>& sh = *reinterpret_cast<FewShared<W>*>(ring_ptr + W * kFewStages * kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = smem_u32(ring_ptr) + (uint32_t)warp * kFewStages * kStage;  // this warp's stages
  if (alone) {
    grid_wait();
  } else {
    if (tid == 0) see_waited(waited);
    __syncthreads();
  }
  grid_launch_dependents();
  // this kernel's end is the end of the one before, too
  const auto leave = [&] {
    grid_wait();
    if (!alone && blockIdx.x == 0 && tid == 0) *waited = 0;
  };

  // ---- this CTA's range of the tile sequence
  FewCursor<W, WIN> c;
  unsigned units = 0, ctas = 0;
  {
    // sums of the tiles over the requests, kThreads at a time; a second
    // round (only with more requests than that) finds the request of the
    // range's first tile
    const bool one = A.requests <= kThreads;
    int u0 = -1;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      long long carry = 0;
#pragma unroll 1
      for (int base = 0; base < A.requests; base += kThreads) {
        c.b = base + tid;
        int tiles = 0;  // of the request, per head
        if (c.b < A.requests) {
          c.take(A, alone);
          if (c.tiles > 0) tiles = c.span() * c.blocks(A);
        }
        long long x = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = x;
        __syncthreads();
        long long at = carry + x - tiles;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (w < warp) at += sh.scan[w];
          carry += sh.scan[w];
        }
        if (u0 < 0 && base + kThreads >= A.requests) {  // the total is known
          const long long total = carry * A.c.kv_heads;
          if (total > INT32_MAX) {
            if (tid == 0) raise_error(A.err, TP3D_EPAGES);
            leave();
            return;
          }
          units = (unsigned)total;
          // kMinTiles tiles each, or an item each where items are shorter (16 heads over 61 keys: 4.7 us, four
          // items to a CTA: 10.3)
          const unsigned items = (unsigned)A.requests * (unsigned)A.c.kv_heads;
          ctas = (units + Shape::kMinTiles - 1) / Shape::kMinTiles;
          ctas = ctas > items ? ctas : items < units ? items : units;
          ctas = ctas < gridDim.x ? ctas : gridDim.x;
          if (blockIdx.x >= ctas) {
            leave();
            return;
          }
          const Ranges R(units, ctas);
          u0 = R.begin(blockIdx.x);
          c.u1 = R.begin(blockIdx.x + 1);
        }
        if (one || round == 1) {
          at *= A.c.kv_heads;
          if (tiles > 0 && at <= u0 && u0 < at + (long long)tiles * A.c.kv_heads) {
            sh.b0 = c.b;
            sh.before = (int)at;
          }
          if (carry * A.c.kv_heads > u0) break;
        }
      }
      if (one) break;
    }
    if (tid < 128) sh.poison[tid] = kNoPoison;
    if (tid == 0) sh.poisoned = 0;
    __syncthreads();
    c.b = sh.b0;
    c.take(A, alone);
    const int off = u0 - sh.before;
    const int item = off / c.span(), blocks = c.blocks(A);
    c.h = c.kBlocks ? item / blocks : item;
    c.row0 = (item - c.h * blocks) * 16;
    const int into = off - item * c.span();
    c.at = u0 - into;
    c.tile = into == 0 ? 0 : c.snap(into);
    if (!(c.tile == c.tiles ? c.next_item(A, alone) : c.share())) {
      leave();
      return;
    }
  }

  const float sl2 = A.scale * kLog2e;
  uint32_t qf[D / 16][4];
  float o[NT][4], m[2], l[2];
  int lim[2];  // the last key that this thread's two rows see
  int low[2];  // the first key of their windows
  FewCursor<W, WIN> ld = c;        // the tile to load next; c: to compute next
  bool begin = true, fetch = true;
  int tile0 = c.tile;      // where this CTA's share of the item begins
  int stage = 0;           // to load into; the next one is the oldest
  int pages = -1, pages_b = -1, pages_at = 0;  // lane i: the page of this warp's keys of tile pages_at + i
#pragma unroll 1
  for (int step = 0;; ++step) {
    // ---- load
    if (fetch) {
      if (ld.b != pages_b || (unsigned)(ld.tile - pages_at) >= 32u) {
        pages_b = ld.b;
        pages_at = ld.tile;
        const int t = ld.tile + lane;
        const int64_t key = (int64_t)(WIN ? ld.gap.tile(t) : t) * kKeys + warp * 16;
        pages = key < ld.kv && !ld.unseen(A, (int)key) ? ld_plain(A.table + (int64_t)ld.b * A.width + (key >> A.page_log2)) : -1;
      }
      const int page = __shfl_sync(0xffffffffu, pages, ld.tile - pages_at);
      const int key = ld.key(ld.tile) + warp * 16, left = ld.kv - key;
      if (left > 0) {
        const bool in = page >= 0 && page < A.c.pages;
        if (!in && !ld.unseen(A, key)) raise_error(A.err, TP3D_EPAGES);
        // lane -> vector (lane % RV) of rows lane / RV + i * (32 / RV); vector v of row r lies at
        // v ^ (r mod 8), so that the eight rows of an 8 x 8 block fall in different banks
        const int v = lane & (RV - 1), r0 = lane / RV;
        const int64_t at = in ? (int64_t)page * A.c.page_stride + (int64_t)((key & (A.c.page - 1)) + r0) * A.c.token_stride +
                                    ld.h * A.c.head_stride + v * 8
                              : 0;
        const bf16* ks = static_cast<const bf16*>(A.c.k) + at;
        const bf16* vs = static_cast<const bf16*>(A.c.v) + at;
        const int64_t hop = in ? (int64_t)(32 / RV) * A.c.token_stride : 0;
        const uint32_t dst = ring + (uint32_t)stage * kStage;
#pragma unroll
        for (int i = 0; i < RV / 2; ++i) {
          const int r = r0 + i * (32 / RV);
          const uint32_t to = dst + (uint32_t)(r * RV + (v ^ (r & 7))) * 16u;
          const bool have = in && r < left && (!WIN || key + r < A.sinks || key + r >= ld.low);
          cp_async16_zfill(to, have ? ks : static_cast<const bf16*>(A.c.k), have);
          cp_async16_zfill(to + kStage / 2, have ? vs : static_cast<const bf16*>(A.c.v), have);
          ks += hop;
          vs += hop;
        }
      }
      fetch = ld.advance(A, alone);
    }
    cp_commit();
    stage = stage == kFewStages - 1 ? 0 : stage + 1;
    if (step < kFewStages - 1) continue;

    // ---- compute the tile in the oldest stage
    const int rows = c.n * A.group - c.row0 < 16 ? c.n * A.group - c.row0 : 16;  // of the block
    if (begin) {
      begin = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = (lane >> 2) + 8 * e;
        const bool in = r < rows;
        const int tok = in ? (c.row0 + r) / A.group : 0, g = in ? c.row0 + r - tok * A.group : 0;
        lim[e] = in ? c.kv - c.n + tok : c.kv - 1;
        if (WIN) low[e] = window_begin(lim[e], A.window);
        const bf16* src = A.q + (c.q0 + tok) * A.q_token + (int64_t)(c.h * A.group + g) * A.q_head + (lane & 3) * 2;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][e] = in ? ld_plain(reinterpret_cast<const uint32_t*>(src + k * 16)) : 0u;
          qf[k][2 + e] = in ? ld_plain(reinterpret_cast<const uint32_t*>(src + k * 16 + 8)) : 0u;
        }
        m[e] = -INFINITY;
        l[e] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    }
    cp_wait<kFewStages - 1>();
    __syncwarp();
    const uint32_t sk = ring + (uint32_t)stage * kStage, sv = sk + kStage / 2;
    const int key0 = c.key(c.tile) + warp * 16;
    if (key0 < c.kv) {
      // keys that some row does not see: past kv - n; before the last row's window
      const int last_low = WIN ? window_begin(c.kv - 1, A.window) : 0;
      const bool partial = key0 + 15 > c.kv - c.n || (WIN && key0 < last_low && key0 + 15 >= A.sinks);
      if (partial && c.n > 1) {
        // A probability of 0 does not silence a value that is not finite: such
        // a value becomes 0, and rows that see its key get NaN in its column
        // at the end.  (Keys that no row sees are zeros in the stage.)
#pragma unroll 1
        for (int i = lane; i < 16 * RV; i += 32) {
          const int r = i / RV, v = i & (RV - 1);
          const uint32_t at = sv + (uint32_t)(r * RV + (v ^ (r & 7))) * 16u;
          const uint4 x = ld_shared4(at);
          __nv_bfloat162 seen = __floats2bfloat162_rn(0.0f, 0.0f);
          watch_finite(seen, x);
          const int k = key0 + r;
          if ((k <= c.kv - c.n && (!WIN || k >= last_low || k < A.sinks)) || !saw_not_finite(seen)) continue;
          int note = k;
          if (WIN) {
            note = 0;
            for (int q = 0; q < rows; ++q) {
              const int p = c.kv - c.n + (c.row0 + q) / A.group;
              if (k <= p && (k >= window_begin(p, A.window) || k < A.sinks)) note |= 1 << q;
            }
          }
          st_shared4(at, make_finite(x, [&](int e) {
                       if (WIN) atomicOr(&sh.poison[v * 8 + e], note);
                       else atomicMin(&sh.poison[v * 8 + e], note);
                     }));
          sh.poisoned = 1;
        }
        __syncwarp();
      }
      // S = Q K^T for 16 keys: two 8-key tiles, two partial sums each
      float s[2][2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][y][e] = 0.0f;
      {
        const int row = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int vec = 2 * k + ((lane >> 3) & 1);
          uint32_t kb[4];
          ldmatrix4(kb, sk + (uint32_t)(row * RV + (vec ^ (row & 7))) * 16u);
          mma16816(s[0][k & 1], qf[k], kb[0], kb[1]);
          mma16816(s[1][k & 1], qf[k], kb[2], kb[3]);
        }
      }
      float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[x][0][e] + s[x][1][e];
          if (partial) {
            const int k = key0 + x * 8 + (lane & 3) * 2 + (e & 1);
            if (k > lim[e >> 1] || (WIN && k < low[e >> 1] && k >= A.sinks)) v = -INFINITY;
          }
          s[x][0][e] = v;
          mt[e >> 1] = fmaxf(mt[e >> 1], v);
        }
      bool move = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], 1));
        mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], 2)) * sl2;
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
      const int row = lane & 15;
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        const int vec = j + (lane >> 4);
        uint32_t vb[4];
        ldmatrix4_trans(vb, sv + (uint32_t)(row * RV + (vec ^ (row & 7))) * 16u);
        mma16816(o[j], ph, vb[0], vb[1]);
        mma16816(o[j + 1], ph, vb[2], vb[3]);
        mma16816(o[j], pl, vb[0], vb[1]);
        mma16816(o[j + 1], pl, vb[2], vb[3]);
      }
    }

    // ---- the item's last tile, or this CTA's: join the warps and write
    if (c.tile + 1 == c.end) {
      const bool whole = tile0 == 0 && c.end == c.tiles;
      // the stage just read takes the warp's O: [row][D], column ^ (row mod 4) * 8 against bank conflicts
      float* const so = reinterpret_cast<float*>(ring_ptr + (size_t)(warp * kFewStages + stage) * kStage);
      __syncthreads();  // (also: every warp's notes are in)
      const bool hurt = sh.poisoned != 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        const int r = (lane >> 2) + 8 * e;
        if ((lane & 3) == 0) {
          sh.m[warp][r] = m[e];
          sh.l[warp][r] = l[e];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int col = j * 8 + (lane & 3) * 2;
          *reinterpret_cast<float2*>(so + r * D + (col ^ ((r & 3) << 3))) = make_float2(o[j][2 * e], o[j][2 * e + 1]);
        }
      }
      __syncthreads();
      // the CTAs whose boundaries lie inside the item and stay there, and the one before them
      const Ranges ranges(units, ctas);
      const int c0 = whole ? 0 : ranges.owner(c.at + Shape::kSnap);
      const int pieces = whole ? 1 : ranges.owner(c.at + c.tiles - Shape::kSnap - 1) - c0 + 1;
      const size_t pf = few_part_floats(D);
      // the part of the item's p-th CTA: an item begins in its CTA's last piece (slot 1), goes on in the
      // next one's first (slot 0); what a group of parts came to (below) has slots of its own
      const auto at = [&](int p) { return parts + ((size_t)(c0 + p) * kFewSlots + (p == 0 ? 1 : 0)) * pf; };
      const auto finish = [&](int r, int col, float4 v, float top, float sum) {
        const int tok = (c.row0 + r) / A.group;
        const int64_t t = c.q0 + tok;
        const int head = c.h * A.group + (c.row0 + r - tok * A.group);
        const float inv = normaliser(sum, c.kv - c.n + tok);
        *reinterpret_cast<uint2*>(A.o + t * A.o_token + (int64_t)head * A.o_head + col) =
            make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
        if (A.lse && col == 0)
          A.lse[t * (int64_t)(A.group * A.c.kv_heads) + head] =
              sum == 0.0f ? -INFINITY : ((top == -INFINITY ? 0.0f : top) + log2f(sum)) * kLn2;
      };
      const auto put = [&](float* to, int r, int col, float4 v, float top, float sum) {
        __stcg(reinterpret_cast<float4*>(to + (size_t)r * D + col), v);
        if (col == 0) {
          __stcg(to + kFewRows * D + r, top);
          __stcg(to + kFewRows * (D + 1) + r, sum);
        }
      };
      const int elems = rows * (D / 4);
#pragma unroll 1
      for (int i = tid; i < elems; i += kThreads) {
        const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, sh.m[w][r]);
        const float tb = top == -INFINITY ? 0.0f : top;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float f = ex2_approx(sh.m[w][r] - tb);
          const float4 v = *reinterpret_cast<const float4*>(so + (w - warp) * (int)(kFewStages * kStage / 4) + r * D +
                                                           (col ^ ((r & 3) << 3)));
          sum += f * sh.l[w][r];
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        if (hurt) {
          const int lr = c.kv - c.n + (c.row0 + r) / A.group;
          float* const x = reinterpret_cast<float*>(&acc);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (WIN ? (sh.poison[col + e] >> r) & 1 : sh.poison[col + e] <= lr) x[e] = __int_as_float(0x7fffffff);
        }
        if (whole) finish(r, col, acc, top, sum);
        else put(at((int)blockIdx.x - c0), r, col, acc, top, sum);
      }
      if (!whole) {
        // Adds parts in order.  Many are joined in two levels: groups of
        // neighbours first, then the groups, so that one CTA never reads them
        // all.  A CTA's arrival may be the last at its group's counter, then
        // at the item's (which so return to zero); one CTA can be an item's
        // first and another's later part: counters of their own.
        const int gsize = pieces <= kJoinOnce ? pieces : (int)ceilf(sqrtf((float)pieces));
        const int groups = (pieces + gsize - 1) / gsize, g = ((int)blockIdx.x - c0) / gsize;
        unsigned* counter = counters + (g == 0 ? 0 : gridDim.x) + c0 + g * gsize;
        const auto group_at = [&](int k) { return parts + ((size_t)(c0 + k * gsize) * kFewSlots + (k == 0 ? 2 : 3)) * pf; };
        const int first = g * gsize;
        int n = pieces - first < gsize ? pieces - first : gsize;
        bool of_groups = false;
#pragma unroll 1
        for (int level = groups == 1 ? 1 : 0; level < 2; ++level) {
          __threadfence();
          __syncthreads();
          if (tid == 0) sh.last = atomicInc(counter, (unsigned)n - 1) == (unsigned)n - 1;
          __syncthreads();
          if (!sh.last) break;
          __threadfence();
          // four parts' maxima, sums and vectors in flight, of two vectors of the result
#pragma unroll 1
          for (int e0 = tid; e0 < elems; e0 += 2 * kThreads) {
            const int e[2] = {e0, e0 + kThreads < elems ? e0 + kThreads : e0};
            const int r[2] = {e[0] / (D / 4), e[1] / (D / 4)};
            float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
            float4 acc[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
#pragma unroll 1
            for (int i0 = 0; i0 < n; i0 += 4) {
              float pm[4][2], ps[4][2];
              float4 pv[4][2];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (i0 + i >= n) break;
                const float* const x = of_groups ? group_at(i0 + i) : at(first + i0 + i);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  pm[i][q] = __ldcg(x + kFewRows * D + r[q]);
                  ps[i][q] = __ldcg(x + kFewRows * (D + 1) + r[q]);
                  pv[i][q] = __ldcg(reinterpret_cast<const float4*>(x) + e[q]);
                }
              }
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float now = top[q];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (i0 + i < n) now = fmaxf(now, pm[i][q]);
                const float base = now == -INFINITY ? 0.0f : now, keep = ex2_approx(top[q] - base);
                sum[q] *= keep;
                acc[q] = make_float4(acc[q].x * keep, acc[q].y * keep, acc[q].z * keep, acc[q].w * keep);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if (i0 + i >= n) break;
                  const float f = ex2_approx(pm[i][q] - base);
                  sum[q] += f * ps[i][q];
                  acc[q].x += f * pv[i][q].x;
                  acc[q].y += f * pv[i][q].y;
                  acc[q].z += f * pv[i][q].z;
                  acc[q].w += f * pv[i][q].w;
                }
                top[q] = now;
              }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (e0 + q * kThreads >= elems) break;
              const int col = (e[q] - r[q] * (D / 4)) * 4;
              if (level == 1) finish(r[q], col, acc[q], top[q], sum[q]);
              else put(group_at(g), r[q], col, acc[q], top[q], sum[q]);
            }
          }
          counter = counters + 2 * gridDim.x + c0;
          of_groups = true;
          n = groups;
        }
      }
      begin = true;
      __syncthreads();  // the stages go back to the loads
      if (hurt) {
        if (tid < 128) sh.poison[tid] = kNoPoison;
        if (tid == 0) sh.poisoned = 0;
        __syncthreads();
      }
    }
    if (!c.advance(A, alone)) break;
    if (begin) tile0 = 0;
  }
  leave();
}

// ------------------------------------------------------------------ many rows
// Requests with more rows per key/value head than that: prompts and their
// chunks.  4 D FLOP per (row, key) pair against 4 D bytes per key: tensor
// work bounds it.  One CTA per SM takes pairs of 128-row query tiles (rows are
// new token x query head of the group, so grouped heads fill a tile with few
// tokens and share its keys) and streams 128-key tiles by TMA, one box per
// page and 64 columns.  As in the layer's forward: S = Q K^T in tensor memory,
// an online softmax per row (one thread each), P written back over S, and
// O += P V with P read from tensor memory.  Differences:
//  * P is kept as two bf16 terms (P = hi + lo up to 2^-16 P): over its 32
//    score columns a chunk leaves 16 columns of hi pairs and 16 of lo pairs,
//    and O += hi V + lo V.  One bf16 term alone has an error as large as the
//    output's own rounding.
//  * The tile sequence (request, head, pair, key tile) is cut into equal
//    contiguous ranges as in the kernel above, so lengths need no plan on the
//    host and every SM gets the same number of tiles.
//  * Key tiles that some row of the pair does not see whole are masked by
//    comparison with each row's last key.  Their values are looked at by two
//    otherwise idle warps before P V: rows past the request become zero, and a
//    value that is not finite becomes zero and is noted with its key and
//    column, since a probability of 0 would not silence it.
//
// Measured: 2048 new tokens over 6145, 16 heads of 128 (120 GFLOP): 141 us in a
// captured graph, 146 us as separate calls: 856 and 824 TFLOP/s, 0.45 and 0.43 of
// the measured bf16 rate; with the lo terms 1.28 and 1.24 PFLOP/s run.
// For D = 128 the tensor instructions bound it: a pair of tiles takes 48 of them,
// 128 x 128 x 16 each, about 107 cycles apiece (64 nominal: two 4 KiB operands
// from shared memory keep its port full), so 5140 of a period of 5250 cycles.
// For D = 64 it is a slot's chain: softmax 2250 cycles, P V 700, S 900 and the
// hand-overs between them make 4400.  A CTA starts its first product 5 us after
// its launch, and a cut item costs 4 us to leave and join.
//
// warps: 0 TMA producer, 1 MMA issuer + TMEM owner, 2-3 value check
// (warpgroup 0); 4-7 slot 0 rows; 8-11 slot 1 rows.
// smem: Q0 | Q1 | R0 .. R4 (a ring of K_j V_j ...), 32 KiB each | barriers | notes
// TMEM: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [256+D,256+2D)
constexpr int kManyThreads = 384;
constexpr int kManyRegsLow = 120, kManyRegsHigh = 192;  // 128 x 120 + 256 x 192 <= 384 x 168 (52 and 68 bytes spilled)
constexpr uint32_t kManyRing = 5;
constexpr int kNotes = 4;  // pieces whose values may be under check or in use at once
struct ManyShared {
  unsigned notes[kNotes][64];    // per column (16 bits): first non-finite masked key - first row's last key
  int noted[kNotes][2];          // by value-check warp
  volatile unsigned ended[8];    // pieces that each row warp has ended: their notes may be begun anew
  int last;
  long long scan[kManyThreads / 32];
  unsigned items;  // pairs of all requests (with a window)
  int before, per_head;
  int b0;
  // split pieces joined after the CTA's range (0: one that it goes on behind, 1: its last): row warps that have
  // left their rows, whether this CTA is to join, the piece's place in the sequence
  int left[2], join[2], place[2][5];
};
constexpr int kManySmem = 7 * (int)kTile + 512 + (int)sizeof(ManyShared) + 1024;
static_assert(kManySmem <= 232448, "shared memory of one CTA");
// Parts of an item joined by row, by the thread that has the CTA's own part in
// tensor memory; more by element, dealt to all row threads.  Up to three by row
// | all by element | up to four by row: 2048 tokens over 6145 keys, 16 heads (2
// parts) 140.6 | 150.0 | 142.4 us; 4 x up to 200 tokens over 3000 (2 to 4) 47.7 |
// 56.2 | 48.0; one prompt of 1000 tokens 31.0 | 35.6 | 29.9.
constexpr int kManyByRow = 3;
constexpr int kManyJoinOnce = 8;  // parts of an item joined in one step (500 tokens over 8192, 5 parts: 74.3 us; with 4 80.4)
constexpr int kManySlots = 4;     // parts that a CTA has room for in the workspace
TP3D_HD constexpr size_t many_part_floats(int d) { return (size_t)2 * TR * (d + 2); }

// sum of floor((a i + b) / TR) for i < n, with a, b < TR; a n + b stays in 32 bits
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t a, uint32_t b) {
  if ((a & (a - 1)) == 0) {  // groups of 2^k heads
    if (a == 0) return 0;
    // a = TR / 2^s: floor((i + floor(b / a)) / 2^s)
    const int s = 7 - (31 - __clz(a));
    const auto upto = [s](int64_t x) {  // sum of floor(i / 2^s) for i < x
      const int64_t q = x >> s;
      return (q * (q - 1) / 2 << s) + q * (x - (q << s));
    };
    const uint32_t off = b >> (7 - s);
    return upto((int64_t)n + off) - upto(off);
  }
  int64_t sum = 0;  // the Euclidean recursion
  uint32_t m = TR;
  while (n > 0) {
    sum += (int64_t)(a / m) * ((int64_t)n * (n - 1) / 2) + (int64_t)(b / m) * n;
    a %= m;
    b %= m;
    const uint32_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const uint32_t t = a;
    a = m;
    m = t;
  }
  return sum;
}

// The pairs of query tiles of a request: pair k holds tokens [2 k tt, +2 tt).
template <bool WIN>
struct ManyRequest {
  int q0, n, kv, tt;  // tt: tokens of a query tile
  int window, sinks;  // (first keys: no more than there are keys)
  __device__ int pairs() const { return (n + 2 * tt - 1) / (2 * tt); }
  // key tiles that tokens below `end` see (one at least: rows without keys are written too)
  __device__ int tiles_upto(int end) const {
    const int keys = kv - n + (end < n ? end : n);
    return keys > 0 ? (keys - 1) / TR + 1 : 1;
  }
  // key tiles that no row of pair k sees, between the first keys and its first row's window
  __device__ Gap gap(int k) const {
    Gap g;
    if (WIN) g.set((sinks + TR - 1) / TR, window_begin(kv - n + k * 2 * tt, window) / TR);
    return g;
  }
  // the same of the pairs before pair k.  Pair i's window begins at c + w i, and what it misses are
  // floor((c + w i) / TR) - lead tiles, from the first pair on where that is positive.
  __device__ int64_t gaps_before(int k) const {
    const int w = 2 * tt, lead = (sinks + TR - 1) / TR;
    const int64_t c = (int64_t)kv - n - window + 1, from = ((int64_t)lead + 1) * TR;
    if (from - c > (int64_t)(k - 1) * w) return 0;
    const int z = c >= from ? 0 : (int)((unsigned)(from - c + w - 1) / (unsigned)w);  // (in 32 bits: k w is)
    const int64_t b = c + (int64_t)w * z, left = k - z;
    return left * (b / TR - lead) + (int64_t)(w / TR) * (left * (left - 1) / 2) +
           floor_sum((uint32_t)left, (uint32_t)(w % TR), (uint32_t)(b % TR));
  }
  __device__ int tiles(int k) const { return tiles_upto((k + 1) * 2 * tt) - gap(k).gap; }
  // key tiles of the pairs before pair k (the last pair's are not among them)
  __device__ int64_t before(int k) const {
    const int w = 2 * tt, ctx = kv - n;
    int z = ctx < 0 ? (int)((unsigned)-ctx / (unsigned)w) : 0;  // pairs whose tokens all see nothing
    if (z > k) z = k;
    const int b = ctx + (z + 1) * w + TR - 1;
    const int64_t left = k - z;
    return z + (int64_t)(b / TR) * left + (int64_t)(w / TR) * (left * (left - 1) / 2) +
           floor_sum((uint32_t)left, (uint32_t)(w % TR), (uint32_t)(b % TR)) - (WIN ? gaps_before(k) : 0);
  }
  __device__ int64_t total() const {
    const int p = pairs();
    return before(p - 1) + tiles(p - 1);
  }
};

template <bool WIN>
__device__ __forceinline__ ManyRequest<WIN> many_request(const PagedAttn& A, int b) {
  const PagedRequest r = paged_request(A, b);
  ManyRequest<WIN> m;
  m.q0 = (int)r.q0;
  m.n = (int64_t)r.n * A.group > A.few_rows ? r.n : 0;  // the others are the kernel above's
  m.kv = r.kv;
  m.tt = TR / A.group;
  if (WIN) {
    m.window = A.window;
    m.sinks = A.sinks < r.kv ? A.sinks : r.kv;
  }
  return m;
}

// One piece of a CTA's range: key tiles [j0, j1) of pair k of (request b, head h).
//
// The pairs of a head come folded - last, first, last but one, second, ... -
// so that neighbours in the sequence add up to like amounts of work, and a
// range boundary within `near` tiles of a pair's edge is moved there: leaving a
// part and joining it costs about as much as kSnap tiles (4 prompts of up to
// 1024: 43.5 us; with 2 43.7, with 1 47.4; 4 x up to 200 tokens over 3000 47.7;
// with 2 52.5; 2048 tokens over 6145 140.6; with 2 139.2).  Where ranges are short, moving by
// as much would leave CTAs without work beside others with twice theirs, so it
// is two tiles less than a range, one at least.  With that | always by kSnap: 4
// requests of 2000 keys, 128 rows a head, 4 heads 26.4 | 30.0 us; 8 chunks of
// up to 100 over 1000, 16 heads of 64 23.2 | 25.8; one prompt of 1000, 16 heads
// 31.0 | 28.5; 4 x 200 over 3000 47.7 | 47.3.
constexpr int kSnap = 4;
// With a window pairs are short, and ranges that end at their edges alone
// unequal.  By two tiles | four | one: 8192 tokens, window 1024, 16 heads of 128
// 123.2 | 131.8 | 124.1 us; 4 x 384 over 3700, window 511, 32 heads of 64 on 8
// 42.4 | 45.5 | 39.3; the same ragged, with 12 single tokens 42.5 | 42.6 | 44.5.
constexpr int kSnapWindow = 2;
// And where pairs are about alike in length and whole ones, dealt out to the CTAs,
// are done no more than kJoin tiles later than equal ranges, none is cut: a cut
// costs its CTAs a piece more to begin and to end, a part to leave and one to
// join.  2048 tokens over 32001, 16 heads of 128, first 4 keys, window 512 37.6 us
// (cut 45.9), 1024 50.7 (56.6), 2048 72.9 (77.9), 4096 108 (108).  With pairs of
// several lengths whole ones come out uneven (4 requests of up to 4084 keys,
// window 1500: 72.8, cut 55.1).
constexpr float kJoin = 4.0f, kAlike = 0.9f;
constexpr int kManyMinTiles = 2;  // of a CTA's range, where there is little work (the first case above; with 1 30.3)
template <bool WIN>
struct ManyCursor {
  ManyRequest<WIN> r;
  Gap gap;          // of the pair
  int low0, low1;   // the pair's key tiles that some row's window leaves out in part: [low0, low1)
  int b, h, i, k, pairs;
  int j0, j1, nkv;  // nkv: the pair's key tiles
  int u, u1;        // the piece's first unit, the range's end (before it is moved)
  int near;         // boundaries this near a pair's edge are moved
  __device__ static int fold(int i, int pairs) { return i & 1 ? i >> 1 : pairs - 1 - (i >> 1); }
  // where a boundary `off` tiles into a pair of n comes to lie
  __device__ int snap(int off, int n) const {
    const int rest = n - off;
    return (off < rest ? off : rest) > near ? off : off <= rest ? 0 : n;
  }
  // enters position i of the folded pairs at tile j0 (unit u): false when the range ends before it
  __device__ bool enter() {
    k = fold(i, pairs);
    nkv = r.tiles(k);
    if (WIN) {
      gap = r.gap(k);
      const int end = (k + 1) * 2 * r.tt < r.n ? (k + 1) * 2 * r.tt : r.n;
      const int last_low = window_begin(r.kv - r.n + end - 1, r.window);  // of the pair's last row
      low0 = gap.at(r.sinks / TR);
      low1 = last_low > r.sinks ? gap.at((last_low - 1) / TR) + 1 : low0;
    }
    const int end = u1 - (u - j0);
    j1 = end >= nkv ? nkv : end > 0 ? snap(end, nkv) : 0;
    return j1 > j0;
  }
  __device__ bool following(const PagedAttn& A) {
    j0 = 0;
    if (u >= u1) return false;
    if (++i == pairs) {
      i = 0;
      if (++h == A.c.kv_heads) {
        h = 0;
        do r = many_request<WIN>(A, ++b);
        while (r.n == 0);
        pairs = r.pairs();
      }
    }
    return enter();
  }
  __device__ bool next(const PagedAttn& A) {
    u += j1 - j0;
    return following(A);
  }
  __device__ int tok(int sl) const { return (2 * k + sl) * r.tt; }  // a slot's first token
  __device__ bool two() const { return tok(1) < r.n; }
  // key tiles of slot sl in this piece
  __device__ int count(int sl) const {
    if (sl) return two() ? j1 - j0 : 0;
    const int n0 = r.tiles_upto(tok(1)) - (WIN ? gap.gap : 0);
    return n0 < j1 ? (n0 > j0 ? n0 - j0 : 0) : j1 - j0;
  }
  __device__ int tile(int j) const { return WIN ? gap.tile(j) : j; }
  // key tile j holds keys that the pair's first row does not see, being behind it
  __device__ bool behind(int j) const { return (tile(j) + 1) * TR - 1 > r.kv - r.n + tok(0); }
  // or that another does not, being before its window
  __device__ bool partial(int j) const { return behind(j) || (WIN && j >= low0 && j < low1); }
  // one of key tiles [a, b) is such a tile
  __device__ bool any_partial(int a, int b) const {
    return behind(b - 1) || (WIN && (a > low0 ? a : low0) < (b < low1 ? b : low1));
  }
};

// How an item cut by range boundaries is joined: its parts are those of CTAs
// [c0, c0 + pieces); groups of gsize of them are joined first, where there are
// many, and then the groups.
struct ManySplit {
  int c0, pieces, gsize, groups;
  template <bool WIN>
  __device__ ManySplit(const ManyCursor<WIN>& cur, unsigned units, unsigned ctas) {
    const Ranges ranges(units, ctas);
    const int item0 = cur.u - cur.j0;
    c0 = ranges.owner(item0 + cur.near);
    pieces = ranges.owner(item0 + cur.nkv - cur.near - 1) - c0 + 1;
    gsize = pieces <= kManyJoinOnce ? pieces : (int)ceilf(sqrtf((float)pieces));
    groups = (pieces + gsize - 1) / gsize;
  }
  __device__ int group() const { return ((int)blockIdx.x - c0) / gsize; }
  __device__ int members(int g) const { return pieces - g * gsize < gsize ? pieces - g * gsize : gsize; }
  // a CTA can be an item's first and another's later part: counters and slots of their own
  __device__ unsigned* counter(unsigned* counters, int g) const {
    return counters + (g == 0 ? 0 : gridDim.x) + c0 + g * gsize;
  }
  __device__ float* part(float* parts, size_t floats, int p) const {
    return parts + ((size_t)(c0 + p) * kManySlots + (p == 0 ? 1 : 0)) * floats;
  }
  __device__ float* group_part(float* parts, size_t floats, int g) const {
    return parts + ((size_t)(c0 + g * gsize) * kManySlots + (g == 0 ? 2 : 3)) * floats;
  }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// 16-bit minimum in a word of two (a rare path: emulated on the word)
__device__ __forceinline__ void note_min(unsigned* word, int half, unsigned v) {
  unsigned old = *reinterpret_cast<volatile unsigned*>(word);
  while (((old >> (16 * half)) & 0xffffu) > v) {
    const unsigned want = half ? (old & 0x0000ffffu) | (v << 16) : (old & 0xffff0000u) | v;
    const unsigned seen = atomicCAS(word, old, want);
    if (seen == old) break;
    old = seen;
  }
}

// One lane of the (converged) warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// 16 columns of a row, scaled and rounded
__device__ __forceinline__ void store_row16(bf16* to, const float* x, float scale) {
  uint32_t p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = pack_bf16(x[2 * e] * scale, x[2 * e + 1] * scale);
  if ((reinterpret_cast<uintptr_t>(to) & 31u) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(p[0]), "r"(p[1]), "r"(p[2]),
                 "r"(p[3]), "r"(p[4]), "r"(p[5]), "r"(p[6]), "r"(p[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(p[0], p[1], p[2], p[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(p[4], p[5], p[6], p[7]);
  }
}

__device__ __forceinline__ void row_warps_meet() { asm volatile("barrier.sync 1, 256;" ::: "memory"); }

// A position in the ring: slot, and the parity of the slot's phase.
struct RingPos {
  uint32_t slot = 0, phase = 0;
  __device__ void next() {
    if (++slot == kManyRing) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// mbar_wait in fewer instructions (the clock and the abort flag are looked at
// after each suspended try): the kernel's roles together fill the instruction
// cache
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, const Ctx& c, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  do {
    if (mbar_try_wait(bar, parity)) return true;
    if (*c.abort_flag) return false;
  } while (globaltimer_ns() - t0 <= wait_limit_ns(err));
  *c.abort_flag = 1;
  raise_error(err, TP3D_ETIMEOUT);
  return false;
}
__device__ __forceinline__ bool warp_wait_on(uint32_t bar, uint32_t parity, const Ctx& c, int* err, int lane) {
  const bool ok = lane == 0 ? wait_on(bar, parity, c, err) : false;
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// The value check goes on to piece p, and may begin its notes, when every row warp has ended
// piece p - kNotes, whose notes lay in their place.  (A slot whose query tile
// is empty does not hold the other up: its row warps may be pieces behind.)
// Bounded as wait_on.
__device__ __forceinline__ bool notes_free(const volatile unsigned* ended, uint32_t piece, const Ctx& c, int* err,
                                           int lane) {
  const auto is = [&] { return __all_sync(0xffffffffu, lane >= 8 || ended[lane & 7] + kNotes > piece) != 0; };
  bool free = is();
  const unsigned long long t0 = free ? 0 : globaltimer_ns();
  while (!free) {
    __nanosleep(200);
    if (__any_sync(0xffffffffu, *c.abort_flag || globaltimer_ns() - t0 > wait_limit_ns(err))) break;
    free = is();
  }
  if (!free && lane == 0 && !*c.abort_flag) {
    *c.abort_flag = 1;
    raise_error(err, TP3D_ETIMEOUT);
  }
  __threadfence_block();
  return free;
}

// One key tile of one row: its 128 scores at `s` in tensor memory become P
// there (per 32 columns: 16 of hi pairs, 16 of lo pairs), the running maximum
// m (base-2 units) and sum l are updated and, when some row of the warp has to
// move its maximum, the row of O at `o` is rescaled.  The first 64 keys' P is
// announced on `half`, so that its product starts while the rest is formed.
// Both passes (maximum, then P) read the scores 32 columns at a time in rolled
// loops: unrolled over the row, the code outgrows the instruction cache and
// runs slower with half the instructions.  What has a paired fp32 form
// (.f32x2) uses it.  PART: only columns up to `vis` are seen.
//
// With a window a pair's first tiles are seen by some of its rows only, and a row
// that has not seen a key yet has an O of zeros (or, after scores of -infinity
// alone, of NaN): its first maximum rescales nothing (2048 tokens over 32001,
// window 6000, 16 heads of 128: 139.5 us against 142.6).
template <int D, bool PART, bool WIN>
__device__ __forceinline__ void many_softmax(uint32_t s, uint32_t o, uint32_t half, int lane, float sl2, int vis,
                                             bool first, float& m, float& l) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int cc = 0; cc < 4; ++cc) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(s + (uint32_t)(cc * 32), v);
    tmem_ld_wait();
    const int left = vis - cc * 32;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float x = !PART || e <= left ? __uint_as_float(v[e]) : -INFINITY;
      const float y = !PART || e + 1 <= left ? __uint_as_float(v[e + 1]) : -INFINITY;
      mx[(e >> 1) & 3] = fmaxf(fmaxf(mx[(e >> 1) & 3], x), y);
    }
  }
  const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
  const bool move = mt > m + kMoveLog2;
  if (__any_sync(0xffffffffu, move)) {
    if (WIN ? __any_sync(0xffffffffu, move && m > -INFINITY) : !first) {
      const float f = move ? ex2_approx(m - mt) : 1.0f;
      l *= f;
#pragma unroll 1
      for (int cc = 0; cc < D / 16; ++cc) {
        uint32_t ov[16];
        tmem_ld_32x32b_x16(o + (uint32_t)(cc * 16), ov);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
        tmem_st_32x32b_x16(o + (uint32_t)(cc * 16), ov);
      }
    }
    if (move) m = mt;
  }
  const float mb = m == -INFINITY ? 0.0f : m;
  const f32x2 sc = splat2(sl2), nb = splat2(-mb), minus = splat2(-1.0f);
  f32x2 sum[4] = {0, 0, 0, 0};
#pragma unroll 1
  for (int cc = 0; cc < 4; ++cc) {
    uint32_t v[32], pk[32];
    tmem_ld_32x32b_x32(s + (uint32_t)(cc * 32), v);
    tmem_ld_wait();
    const int left = vis - cc * 32;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float p0, p1, t0, t1;
      upk2(fma2(pk2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sc, nb), p0, p1);
      p0 = !PART || 2 * e <= left ? ex2_approx(p0) : 0.0f;
      p1 = !PART || 2 * e + 1 <= left ? ex2_approx(p1) : 0.0f;
      const f32x2 P = pk2(p0, p1);
      sum[e & 3] = add2(sum[e & 3], P);
      // hi: the upper halves as they are (truncated to bf16); lo: the exact rest, rounded
      const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
      pk[e] = __byte_perm(b0, b1, 0x7632);
      upk2(fma2(pk2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u)), minus, P), t0, t1);
      pk[16 + e] = pack_bf16(t0, t1);
    }
    tmem_st_32x32b_x32(s + (uint32_t)(cc * 32), pk);
    if (cc == 1) {
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(half, lane);
    }
  }
  tmem_st_wait();
  float a0, a1;
  upk2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a0, a1);
  l += a0 + a1;
}

// With a window, the scores of a tile that a row does not see become -infinity
// where they lie, and the softmax is that of whole tiles: of a warp's four groups
// of 32 columns mostly one is seen in part, and a second softmax's instructions
// would have to be fetched for every tile at a window's edge (8192 tokens, window
// 1024, 16 heads of 64: 102.1 us, with one 104.5; 2048 over 32001, window 4096,
// heads of 128: 106.0, 107.6).  Seen are the columns up to `vis` and from `from`
// on, and those below `upto`.
struct Seen {
  int vis, from, upto;
  // of columns [c, c + 32), a bit each
  __device__ uint32_t bits(int c) const { return below(vis + 1 - c) & (~below(from - c) | below(upto - c)); }
  __device__ static uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
};
__device__ __forceinline__ void hide_unseen(uint32_t s, const Seen& seen) {
#pragma unroll 1
  for (int cc = 0; cc < 4; ++cc) {
    const uint32_t in = seen.bits(cc * 32);
    if (__all_sync(0xffffffffu, in == ~0u)) continue;
    uint32_t v[32];
    tmem_ld_32x32b_x32(s + (uint32_t)(cc * 32), v);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = in >> e & 1u ? v[e] : 0xff800000u;
    tmem_st_32x32b_x32(s + (uint32_t)(cc * 32), v);
  }
  tmem_st_wait();
}

// With a window, which rows see a key is an interval of its own for each key,
// so the row of new token `token` looks for the values that the check has set to
// zero itself: at the keys that it sees in the first `cnt` tiles of the piece, of
// those tiles that were checked.  Returns the columns of [col, col + N) that have
// one, a bit each.  Only where the check has found a value that is not finite.
template <bool WIN, int N>
__device__ __noinline__ uint32_t spoilt(const PagedAttn& A, const ManyCursor<WIN>& at, int cnt, int token, int col) {
  const int lim = at.r.kv - at.r.n + token, low = window_begin(lim, at.r.window);
  uint32_t bits = 0;
  if (token >= at.r.n) return bits;
#pragma unroll 1
  for (int j = at.j0; j < at.j0 + cnt; ++j) {
    if (!at.partial(j)) continue;
#pragma unroll 1
    for (int key = at.tile(j) * TR; key < (at.tile(j) + 1) * TR && key <= lim; ++key) {
      if (key < low && key >= at.r.sinks) continue;
      const int32_t page = ld_plain(A.table + (int64_t)at.b * A.width + (key >> A.page_log2));
      if (page < 0 || page >= A.c.pages) continue;
      const bf16* const v = static_cast<const bf16*>(A.c.v) + page * A.c.page_stride +
                            (key & (A.c.page - 1)) * A.c.token_stride + at.h * A.c.head_stride + col;
#pragma unroll
      for (int q = 0; q < N / 8; ++q) {
        const uint4 x = ld_plain(reinterpret_cast<const uint4*>(v) + q);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((w[e >> 1] >> (16 * (e & 1)) & 0x7f80u) == 0x7f80u) bits |= 1u << (8 * q + e);
      }
    }
  }
  return bits;
}

template <int D, bool WIN>
__global__ void __launch_bounds__(kManyThreads, 1)
    paged_attn_many_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const PagedAttn A, float* __restrict__ parts,
                           unsigned* __restrict__ counters, unsigned* waited) {
  constexpr int NCH = D / 64;
  extern __shared__ uint8_t smem_raw[];
  grid_wait();
  if (waited && blockIdx.x == 0 && threadIdx.x == 0) say_waited(waited);
  grid_launch_dependents();
  const Ctx c = setup_smem(smem_raw);
  ManyShared& sh = *reinterpret_cast<ManyShared*>(c.base_ptr + 7 * kTile + 512);
  auto sQ = [&](int sl) { return c.base + (uint32_t)sl * kTile; };
  auto sR = [&](uint32_t i) { return c.base + (2u + i) * kTile; };
  auto bar = [&](int k) { return c.bar0 + 8u * k; };
  const uint32_t q_full = bar(0), q_empty = bar(1), final_bar = bar(22), part_full = bar(28), part_last = bar(29);
  auto r_full = [&](uint32_t i) { return bar(2 + (int)i); };
  auto r_empty = [&](uint32_t i) { return bar(2 + (int)kManyRing + (int)i); };
  auto s_full = [&](int sl) { return bar(12 + sl); };
  auto p_full = [&](int sl) { return bar(14 + sl); };
  auto p_empty = [&](int sl) { return bar(16 + sl); };
  auto o_full = [&](int sl) { return bar(18 + sl); };
  auto o_empty = [&](int sl) { return bar(20 + sl); };
  auto p_half = [&](int sl) { return bar(30 + sl); };
  auto v_checked = [&](uint32_t i) { return bar(23 + (int)i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- this CTA's range of the tile sequence (as in the kernel above)
  unsigned units = 0, ctas = 0;
  ManyCursor<WIN> cur;
  {
    const bool one = A.requests <= kManyThreads;
    cur.u = -1;
    unsigned items = 0;
    if (WIN && threadIdx.x == 0) sh.items = 0;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      long long carry = 0;
#pragma unroll 1
      for (int base = 0; base < A.requests; base += kManyThreads) {
        const int b = base + (int)threadIdx.x;
        long long tiles = 0;
        if (b < A.requests) {
          const ManyRequest<WIN> r = many_request<WIN>(A, b);
          if (r.n > 0) {
            tiles = r.total();
            if (WIN && round == 0) items += (unsigned)r.pairs();
          }
        }
        long long x = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = x;
        __syncthreads();
        long long at = carry + x - tiles;
#pragma unroll 4
        for (int w = 0; w < kManyThreads / 32; ++w) {
          if (w < warp) at += sh.scan[w];
          carry += sh.scan[w];
        }
        if (cur.u < 0 && base + kManyThreads >= A.requests) {  // the total is known
          const long long total = carry * A.c.kv_heads;
          if (total > INT32_MAX) {
            if (threadIdx.x == 0) raise_error(A.err, TP3D_EPAGES);
            return;
          }
          units = (unsigned)total;
          ctas = (units + kManyMinTiles - 1) / kManyMinTiles;
          ctas = ctas < gridDim.x ? ctas : gridDim.x;
          if (blockIdx.x >= ctas) return;
          const Ranges R(units, ctas);
          cur.u = R.begin(blockIdx.x);
          const int near = (int)(units / ctas) - 2;
          constexpr int most = WIN ? kSnapWindow : kSnap;
          cur.near = near < 1 ? 1 : near < most ? near : most;
          if (WIN) {
            items = __reduce_add_sync(0xffffffffu, items);
            if (lane == 0) atomicAdd(&sh.items, items);
            __syncthreads();
            const float range = (float)units / (float)ctas;
            const float pair = (float)units / ((float)sh.items * (float)A.c.kv_heads);
            const float longest = (float)A.window / TR + (float)A.sinks / TR + (float)(2 * (TR / A.group)) / TR + 2.0f;
            if (pair >= kAlike * longest && ceilf(range / pair) * pair <= range + kJoin) cur.near = INT32_MAX / 2;
          }
          cur.u1 = R.begin(blockIdx.x + 1);
          if (cur.u >= cur.u1) return;
        }
        if (one || round == 1) {
          at *= A.c.kv_heads;
          if (tiles > 0 && at <= cur.u && cur.u < at + tiles * A.c.kv_heads) {
            sh.b0 = b;
            sh.before = (int)at;
            sh.per_head = (int)tiles;
          }
          if (carry * A.c.kv_heads > cur.u) break;
        }
      }
      if (one) break;
    }
  }
  __syncthreads();
  cur.b = sh.b0;
  cur.r = many_request<WIN>(A, cur.b);
  cur.pairs = cur.r.pairs();
  {
    const int per_head = sh.per_head;
    int off = cur.u - sh.before;
    cur.h = off / per_head;
    off -= cur.h * per_head;
    // the last position of the folded pairs that begins at or before `off`:
    // 32 candidates at a time, one a lane.  Before position i lie the tiles of
    // the last (i + 1) / 2 pairs and of the first i / 2.
    int lo = 0, hi = cur.pairs, begins = 0;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      int at = 0;
      if (i > 0 && i < hi) {
        at = per_head;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {  // (one copy of the instructions: they are fetched for the first time here)
          const int t = (int)cur.r.before(e ? i / 2 : cur.pairs - (i + 1) / 2);
          at += e ? t : -t;
        }
      }
      const int n = __popc(__ballot_sync(0xffffffffu, i < hi && at <= off));  // one at least: lo itself
      begins = __shfl_sync(0xffffffffu, at, n - 1);
      lo += (n - 1) * step;
      hi = lo + step < hi ? lo + step : hi;
    }
    cur.i = lo;
    const int into = off - begins, n = cur.r.tiles(ManyCursor<WIN>::fold(lo, cur.pairs));
    cur.j0 = into == 0 ? 0 : cur.snap(into, n);
    cur.u += cur.j0 - into;
    if (!(cur.j0 == n ? cur.following(A) : cur.enter())) return;
  }
  if (threadIdx.x == 0) {
    for (int k = 0; k < 32; ++k) {
      // p_half, p_full, o_empty: one arrival per row warp of the slot; r_empty: the
      // issuer and the two value-check warps (which follow every slot, so that
      // no phase passes them by); v_checked: those two; part_full: all row warps
      const bool four = k == 14 || k == 15 || k == 20 || k == 21 || k >= 30, ring_empty = k >= 7 && k < 12;
      mbar_init(bar(k), four ? 4 : ring_empty ? 3 : k >= 23 && k < 28 ? 2 : k == 28 ? 8 : 1);
    }
    *c.abort_flag = 0;
    sh.left[0] = sh.left[1] = sh.join[0] = sh.join[1] = 0;
    for (int w = 0; w < 8; ++w) sh.ended[w] = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&mq);
    tma_prefetch_map(&mk);
    tma_prefetch_map(&mv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(c.tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *c.tmem_holder;
  if (warp < 4) {
    // ---------------------------------------------------------- warpgroup 0
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kManyRegsLow));
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      // lane -> (page of the tile, 64-column chunk): one box each
      const int bl2 = A.page_log2 < 7 ? A.page_log2 : 7;  // a box's keys
      const int boxes = TR >> bl2;
      const int pi = lane & (boxes - 1), ch = lane / boxes;
      const bool mine = ch < NCH;
      const uint32_t box_dst = (uint32_t)ch * kChunk + ((uint32_t)pi << bl2) * 128u;
      const uint32_t kv_bytes = (uint32_t)TR * D * 2, q_bytes = (uint32_t)(cur.r.tt * A.group) * D * 2;
      RingPos pos;
      uint32_t n = 0, ic = 0;
      bool ok = true;
      do {
        const bool two = cur.two();
        if (!(ok = warp_wait_on(q_empty, (ic & 1) ^ 1, c, A.err, lane))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, q_bytes * (two ? 2u : 1u));
          for (int sl = 0; sl < (two ? 2 : 1); ++sl)
            for (int x = 0; x < NCH; ++x)
              tma_load_3d(sQ(sl) + (uint32_t)x * kChunk, &mq, q_full, 64 * x, cur.h * A.group,
                          cur.r.q0 + cur.tok(sl));
        }
        ++ic;
        for (int j = cur.j0; j < cur.j1 && ok; ++j) {
          // a box outside the request or the pool starts past the last page: TMA fills it with zeros; one whose keys
          // no row of the pair sees, too (its page may have been given back)
          const int key = cur.tile(j) * TR + (pi << bl2);
          int32_t page = (int32_t)A.c.pages;
          const bool unseen = WIN && key >= cur.r.sinks &&
                              key + (1 << bl2) <= window_begin(cur.r.kv - cur.r.n + cur.tok(0), cur.r.window);
          if (mine && key < cur.r.kv && !unseen) {
            page = ld_plain(A.table + (int64_t)cur.b * A.width + (key >> A.page_log2));
            if (page < 0 || page >= A.c.pages) {
              raise_error(A.err, TP3D_EPAGES);
              page = (int32_t)A.c.pages;
            }
          }
          const int in_page = (int)(key & (A.c.page - 1));
          for (int kvi = 0; kvi < 2; ++kvi, ++n, pos.next()) {
            const uint32_t slot = pos.slot;
            // test hook: stop loading (and let what is in flight land, below)
            if (A.stall_after >= 0 && (int64_t)n >= A.stall_after) {
              ok = false;
              break;
            }
            if (!(ok = warp_wait_on(r_empty(slot), pos.phase ^ 1, c, A.err, lane))) break;
            if (lane == 0) mbar_arrive_expect_tx(r_full(slot), kv_bytes);
            __syncwarp();
            if (mine) tma_load_4d(sR(slot) + box_dst, kvi ? &mv : &mk, r_full(slot), 64 * ch, in_page, cur.h, page);
          }
        }
      } while (ok && cur.next(A));
      if (lane == 0) {  // let what was issued land before the CTA's shared memory goes, whether or not it is waited for
        if (ic) drain(q_full, (ic - 1) & 1);
        for (uint32_t i = n > kManyRing ? n - kManyRing : 0; i < n; ++i)
          drain(r_full(i % kManyRing), (i / kManyRing) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp walks the loop and one elected lane issues: descriptors
      // and addresses then live in uniform registers, which the tensor
      // instructions take directly (from a lane's own registers every one of
      // them is moved over first, and the products no longer follow each other
      // without a pause).  What the loop needs of a piece is broadcast once.
      constexpr uint32_t id_s = idesc_bf16_f32(TR, TR, 0, 0);  // S = Q K^T
      constexpr uint32_t id_o = idesc_bf16_f32(TR, D, 0, 1);   // O += P V (P from TMEM, V MN-major)
      constexpr uint64_t kSlotStep = kTile >> 4;
      const uint32_t ubase = __shfl_sync(0xffffffffu, c.base, 0), utmem = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = desc_kmajor(ubase, 0), k_desc = desc_kmajor(ubase + 2 * kTile, 0),
                     v_desc = desc_mnmajor(ubase + 2 * kTile, 0);
      RingPos pos;
      uint32_t ic = 0, vc = 0;  // vc: the next v_checked phase's parity, a bit per slot
      uint32_t pc[2] = {0, 0}, oc[2] = {0, 0};  // P V products issued, pieces finished, per slot
      bool ok = true;
      // Every lane waits by its own clock, so a wait may run out for one lane
      // and not for another.  No lane leaves the others alone with instructions
      // of the whole warp: all go on, over tiles that may not be there (their
      // results no longer count, and what they touch stays the CTA's), and one
      // vote on the abort flag per key tile ends the loop for all.  (A vote per
      // wait: 2048 tokens over 6145 146.7 us against 140.6.)
      auto wait = [&](uint32_t b, uint32_t parity) {
        wait_on(b, parity, c, A.err);
      };
      auto commit = [&](uint32_t b) {
        if (elect_one()) umma_commit(b);
      };
      auto issue_s = [&](int sl, uint32_t kslot) {
        if (pc[sl] > 0) wait(p_empty(sl), (pc[sl] - 1) & 1);
        tc_fence_after();
        const uint64_t qd = q_desc + (uint64_t)sl * kSlotStep, kd = k_desc + kslot * kSlotStep;
        const uint32_t st = utmem + (uint32_t)(sl * TR);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t step = (uint64_t)((k >> 2) * (kChunk >> 4) + (k & 3) * 2);
            umma_bf16(st, qd + step, kd + step, id_s, k > 0 ? 1u : 0u);
          }
          umma_commit(s_full(sl));
        }
      };
      auto issue_pv = [&](int sl, uint32_t vslot, bool first) {
        const uint32_t pt = utmem + (uint32_t)(sl * TR), ot = utmem + 256u + (uint32_t)(sl * D);
        const uint64_t vd = v_desc + vslot * kSlotStep;
        if (first) wait(o_empty(sl), (oc[sl] & 1) ^ 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wait(h ? p_full(sl) : p_half(sl), pc[sl] & 1);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = h * TR / 32; k < (h + 1) * TR / 32; ++k) {
              const uint32_t hi = pt + (uint32_t)(32 * (k >> 1) + 8 * (k & 1));
              umma_ts(ot, hi, vd + (uint64_t)(k * 128), id_o, k > 0 || !first ? 1u : 0u);
              umma_ts(ot, hi + 16u, vd + (uint64_t)(k * 128), id_o, 1u);
            }
            if (h) umma_commit(p_empty(sl));
          }
        }
        ++pc[sl];
      };
      do {
        const int cnt[2] = {__shfl_sync(0xffffffffu, cur.count(0), 0), __shfl_sync(0xffffffffu, cur.count(1), 0)};
        const int nmax = __shfl_sync(0xffffffffu, cur.j1 - cur.j0, 0);
        // the first key tile of the piece that some row does not see whole
        const int seen = cur.r.kv - cur.r.n + cur.tok(0) + 1;
        const int seen_tiles = seen > 0 ? seen / TR : 0;
        const int part0 = __shfl_sync(0xffffffffu, (WIN ? cur.gap.at(seen_tiles) : seen_tiles) - cur.j0, 0);
        // those that some row's window leaves out in part
        const int low0 = WIN ? __shfl_sync(0xffffffffu, cur.low0 - cur.j0, 0) : 0;
        const int low1 = WIN ? __shfl_sync(0xffffffffu, cur.low1 - cur.j0, 0) : 0;
        // the value tile of key tile i of the piece, in and (where some row does not see it whole) checked
        auto values = [&](int i, uint32_t& vs) {
          vs = pos.slot;
          wait(r_full(vs), pos.phase);
          pos.next();
          if (i < part0 && (!WIN || i < low0 || i >= low1)) return;
          wait(v_checked(vs), (vc >> vs) & 1);
          vc ^= 1u << vs;
        };
        wait(q_full, ic & 1);
        wait(r_full(pos.slot), pos.phase);
        ++ic;
        uint32_t ks = pos.slot, vs = 0, vn = 0;
        pos.next();
        if (cnt[0] > 0) issue_s(0, ks);
        if (cnt[1] > 0) issue_s(1, ks);
        if (nmax == 1) commit(q_empty);
        commit(r_empty(ks));
        values(0, vs);
        // P0 V, S0 of the next tile, P1 V, S1 of the next tile; a slot's next S
        // waits for its P V (it overwrites P), and what else the next tile
        // needs is waited for in the shadow of that
        for (int i = 0; i < nmax; ++i) {
          const bool more = i + 1 < nmax;
          if (i < cnt[0]) issue_pv(0, vs, i == 0);
          // Its rows go on to their output while the other slot ends (prompts 4 x up to 1024 43.5 -> 43.0 us; the
          // windowed chunk of 2048 106.0 -> 104.1).
          if (i + 1 == cnt[0]) {
            commit(o_full(0));
            ++oc[0];
          }
          const int aborted = *c.abort_flag;
          if (more) {
            ks = pos.slot;
            wait(r_full(ks), pos.phase);
            pos.next();
            if (i + 1 < cnt[0]) issue_s(0, ks);
          }
          if (i < cnt[1]) issue_pv(1, vs, i == 0);
          commit(r_empty(vs));
          if (more) {
            values(i + 1, vn);
            if (i + 1 < cnt[1]) issue_s(1, ks);
            commit(r_empty(ks));
            if (i + 2 == nmax) commit(q_empty);  // the piece's last product with Q issued
            vs = vn;
          }
          if (__any_sync(0xffffffffu, aborted)) {
            ok = false;
            break;
          }
        }
        if (!ok) break;
        if (cnt[1] > 0) {
          commit(o_full(1));
          ++oc[1];
        }
      } while (cur.next(A));
      commit(final_bar);
      drain(final_bar, 0);
    } else if (warp >= 2) {
      // ------------------------------------------------------------ value check
      // warp w looks at half of the columns of each partly seen value tile:
      // 16-byte vectors [w * NV, +NV) of the row's D / 8
      constexpr int NV = D / 16;
      const int w = warp - 2;
      RingPos pos;
      uint32_t ic = 0;
      bool ok = true;
      do {
        if (!(ok = notes_free(sh.ended, ic, c, A.err, lane))) break;
        const int seen = cur.r.kv - cur.r.n + cur.tok(0);  // the first row's last key
        unsigned* const notes = sh.notes[ic % kNotes] + w * (NV * 4);
        bool noting = false;
        for (uint32_t i2 = 0; i2 < 2 * (uint32_t)(cur.j1 - cur.j0); ++i2, pos.next()) {
          const int j = cur.j0 + (int)(i2 >> 1);
          const uint32_t slot = pos.slot;
          if (!(ok = warp_wait_on(r_full(slot), pos.phase, c, A.err, lane))) break;
          if (!(i2 & 1) || !cur.partial(j)) {
            warp_arrive(r_empty(slot), lane);
            continue;
          }
          if (!noting) {
            noting = true;
            if (!WIN)
              for (int i = lane; i < NV * 4; i += 32) notes[i] = 0xffffffffu;
            if (lane == 0) sh.noted[ic % kNotes][w] = 0;
            __syncwarp();
          }
          // (with a window, any key of the tile: what is not finite becomes zero, and the rows look for it themselves)
          const int k0 = cur.tile(j) * TR, from = !WIN && seen + 1 > k0 ? seen + 1 - k0 : 0;
          constexpr int RG = 32 / NV;  // rows per step of the warp
          const int v = w * NV + (lane & (NV - 1)), row = lane / NV;
          const uint32_t col = sR(slot) + (uint32_t)(v >> 3) * kChunk;
          const auto at = [&](int key) { return col + (uint32_t)(key * 128 + (((v & 7) ^ (key & 7)) << 4)); };
          // rows past the request: zero
          const int end = cur.r.kv - k0 < TR ? cur.r.kv - k0 : TR;
#pragma unroll 1
          for (int key = (end > 0 ? end : 0) + row; key < TR; key += RG) st_shared4(at(key), make_uint4(0, 0, 0, 0));
          __nv_bfloat162 sum0 = __floats2bfloat162_rn(0.0f, 0.0f);
          // rows 8 apart are 1024 bytes apart; eight loads in flight, since the
          // tensor core's own reads of shared memory hold each of them up
#pragma unroll 1
          for (int key = from + row; key < from + row + 8; key += RG) {
            const uint32_t p = at(key);
#pragma unroll 1
            for (int m = 0; key + 8 * m < end; m += 8) {
              uint4 x[8];
#pragma unroll
              for (int q = 0; q < 8; ++q)
                x[q] = key + 8 * (m + q) < end ? ld_shared4(p + 1024u * (uint32_t)(m + q)) : make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int q = 0; q < 8; ++q) watch_finite(sum0, x[q]);
            }
          }
          if (__any_sync(0xffffffffu, saw_not_finite(sum0))) {
#pragma unroll 1
            for (int key = from + row; key < end; key += RG) {
              const unsigned rel = (unsigned)(k0 + key - seen < 0xfffe ? k0 + key - seen : 0xfffe);
              st_shared4(at(key), make_finite(ld_shared4(at(key)), [&](int i) {
                           if (!WIN) note_min(notes + (v - w * NV) * 4 + (i >> 1), i & 1, rel);
                         }));
            }
            if (lane == 0) sh.noted[ic % kNotes][w] = 1;
          }
          fence_proxy_async_smem();  // the tensor core reads what was rewritten
          warp_arrive(v_checked(slot), lane);
          warp_arrive(r_empty(slot), lane);
        }
        ++ic;
      } while (ok && cur.next(A));
    }
  } else {
    // ------------------------------------------------------------ softmax rows (warpgroups 1, 2)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegsHigh));
    const int sl = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // the slot's row: token r / group, head r % group
    const int tok = r / A.group, g = r - tok * A.group;
    const float sl2 = A.scale * kLog2e;
    const uint32_t s_col = (uint32_t)(sl * TR), o_col = 256u + (uint32_t)(sl * D);
    const size_t pf = many_part_floats(D);
    uint32_t sc = 0, oc = 0, ic = 0;  // score tiles, finished accumulators, pieces
    uint32_t xc = 0;                  // questions about split pieces
    bool ok = true, more = true;
    // of the piece just finished (the last one's are used after the loop)
    ManyCursor<WIN> at = cur;
    float m = -INFINITY, l = 0.0f;
    int cnt = 0;
    bool live = false, hurt = false, by_row = false, last = false;
    // columns whose notes say that this row sees a value that is not finite
    const auto spoil = [&](auto& ov, int col) {
      if (WIN) {
        constexpr int N = (int)(sizeof(ov) / 4);
        const ManyCursor<WIN> piece = at;  // (a copy in memory for the call)
        const uint32_t bits = spoilt<WIN, N>(A, piece, cnt, piece.tok(sl) + tok, col);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (bits >> e & 1u) ov[e] = 0x7fffffffu;
        return;
      }
      const unsigned* const notes = sh.notes[ic % kNotes];
      const unsigned rel = (unsigned)(at.tok(sl) + tok - at.tok(0));  // the row's last key - the pair's first row's
#pragma unroll
      for (int e = 0; e < (int)(sizeof(ov) / 4); ++e)
        if (((notes[(col + e) >> 1] >> (16 * (e & 1))) & 0xffffu) <= rel) ov[e] = 0x7fffffffu;
    };
    const auto put_lse = [&](int64_t row, int head, float top, float sum) {
      if (A.lse)
        A.lse[row * (int64_t)(A.group * A.c.kv_heads) + head] =
            sum == 0.0f ? -INFINITY : ((top == -INFINITY ? 0.0f : top) + log2f(sum)) * kLn2;
    };
    // All row warps meet, one asks, and all hear the answer: `count` is whether
    // the CTA arrives at the item's count (which returns to zero with the last
    // arrival) or only looks whether it would be the last.
    const auto ask = [&](bool count, unsigned* counter, int of, bool& answer) -> bool {
      warp_arrive(part_full, lane);
      if (warp == 4 && lane == 0 && wait_on(part_full, xc & 1, c, A.err)) {
        if (count) {
          __threadfence();
          sh.last = atomicInc(counter, (unsigned)of - 1) == (unsigned)of - 1;
        } else {
          sh.last = counter_load_acquire(reinterpret_cast<const int*>(counter)) == of - 1;
          if (sh.last) *counter = 0;
        }
        mbar_arrive(part_last);
      }
      if (!warp_wait_on(part_last, xc & 1, c, A.err, lane)) return false;
      ++xc;
      answer = *reinterpret_cast<volatile int*>(&sh.last) != 0;
      return true;
    };
    do {
      cnt = cur.count(sl);
      const int token = cur.tok(sl) + tok;  // of the request
      live = tok < cur.r.tt && token < cur.r.n;
      const int lim = cur.r.kv - cur.r.n + token;  // the row's last key
      m = -INFINITY;
      l = 0.0f;
      for (int j = cur.j0; j < cur.j0 + cnt && ok; ++j) {
        // new scores; they also mean the slot's previous P V has finished
        if (!(ok = warp_wait_on(s_full(sl), sc & 1, c, A.err, lane))) break;
        ++sc;
        tc_fence_after();
        // columns of this tile that the row sees: [0, vis]
        const int k0 = cur.tile(j) * TR;
        const int vis = lim - k0;
        const uint32_t sa = tmem_row(tmem, quarter, s_col), oa = tmem_row(tmem, quarter, o_col);
        if (WIN) {
          const Seen seen{vis, window_begin(lim, A.window) - k0, cur.r.sinks - k0};
          if (__any_sync(0xffffffffu, vis < TR - 1 || (seen.from > 0 && seen.upto < TR))) hide_unseen(sa, seen);
          many_softmax<D, false, WIN>(sa, oa, p_half(sl), lane, sl2, vis, j == cur.j0, m, l);
        } else if (__any_sync(0xffffffffu, vis < TR - 1)) {
          many_softmax<D, true, WIN>(sa, oa, p_half(sl), lane, sl2, vis, j == cur.j0, m, l);
        } else {
          many_softmax<D, false, WIN>(sa, oa, p_half(sl), lane, sl2, vis, j == cur.j0, m, l);
        }
        tc_fence_before();
        warp_arrive(p_full(sl), lane);
      }
      if (!ok) break;
      if (cnt > 0) {
        if (!(ok = warp_wait_on(o_full(sl), oc & 1, c, A.err, lane))) break;
        ++oc;
        tc_fence_after();
      }
      hurt = cnt > 0 && cur.any_partial(cur.j0, cur.j0 + cnt) && (sh.noted[ic % kNotes][0] | sh.noted[ic % kNotes][1]) != 0;
      at = cur;
      more = cur.next(A);
      if (at.j0 == 0 && at.j1 == at.nkv) {
        const float inv = normaliser(l, lim);
        const int64_t row = (int64_t)at.r.q0 + token;
        const int head = at.h * A.group + g;
        bf16* const dst = A.o + row * A.o_token + (int64_t)head * A.o_head;
        if (cnt > 0) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t ov[32];
            tmem_ld_32x32b_x32(tmem_row(tmem, quarter, o_col + (uint32_t)(cc * 32)), ov);
            tmem_ld_wait();
            if (hurt) spoil(ov, cc * 32);
            if (live) store_row32(dst + cc * 32, ov, inv);
          }
        }
        if (live) put_lse(row, head, m, l);
      } else {
        // The CTAs whose boundaries lie inside the item and stay there, and the
        // one before them, each have a part of it, and leave it in the
        // workspace: element (column block of 4, row), rows consecutive, so
        // that a warp's accesses are.
        const ManySplit split(at, units, ctas);
        // Few parts: the last CTA to come adds them, its own out of tensor
        // memory, each row by its thread.  It is nearly always one whose range
        // ends here, and where all others have left theirs before it looks, its
        // part need not be written at all.  Where the range goes on, no warp
        // waits for an answer, and in case it was the last the joining is put
        // off until after the range.
        by_row = !more && split.pieces <= kManyByRow;
        if (by_row && !(ok = ask(false, counters + split.c0, split.pieces, last))) break;
        if (last) break;
        float* const part = split.part(parts, pf, (int)blockIdx.x - split.c0);
        const int prow = sl * TR + r;
        if (cnt > 0) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t ov[32];
            tmem_ld_32x32b_x32(tmem_row(tmem, quarter, o_col + (uint32_t)(cc * 32)), ov);
            tmem_ld_wait();
            if (hurt) spoil(ov, cc * 32);
            if (live)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                __stcg(reinterpret_cast<uint4*>(part) + (size_t)(cc * 8 + e) * (2 * TR) + prow,
                       make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]));
          }
        }
        if (live) {
          __stcg(part + (size_t)2 * TR * D + prow, m);
          __stcg(part + (size_t)2 * TR * (D + 1) + prow, cnt > 0 ? l : -1.0f);  // -1: no O has been left
        }
        if (by_row) break;
        __syncwarp();
        const int which = more ? 0 : 1;
        if (lane == 0) {
          __threadfence_block();
          if (atomicAdd(&sh.left[which], 1) == 7) {  // the last row warp arrives for the CTA
            __threadfence();
            const int gr = split.group();
            const unsigned n = (unsigned)split.members(gr);
            sh.join[which] = atomicInc(split.counter(counters, gr), n - 1) == n - 1;
            int* const place = sh.place[which];
            place[0] = at.b;
            place[1] = at.h;
            place[2] = at.k;
            place[3] = at.nkv;
            place[4] = at.u - at.j0;
          }
        }
      }
      if (cnt > 0) {
        tc_fence_before();
        warp_arrive(o_empty(sl), lane);
      }
      ++ic;
      if (lane == 0) {
        __threadfence_block();
        sh.ended[warp - 4] = ic;
      }
    } while (more);
    if (ok && by_row) {
      const ManySplit split(at, units, ctas);
      const int own = (int)blockIdx.x - split.c0, prow = sl * TR + r;
      if (!last) ok = ask(true, counters + split.c0, split.pieces, last);
      if (ok && last) {
        __threadfence();
        const int64_t row = (int64_t)at.r.q0 + at.tok(sl) + tok;
        const int head = at.h * A.group + g;
        bf16* const dst = A.o + row * A.o_token + (int64_t)head * A.o_head;
        // the weights of this row's parts first (a sum below 0: there is no O)
        constexpr int kOthers = kManyByRow - 1;
        const auto other = [&](int i) { return split.part(parts, pf, i + (i >= own ? 1 : 0)); };
        float om[kOthers], ol[kOthers], top = m, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kOthers; ++i) {
          const bool in = live && i < split.pieces - 1;
          om[i] = in ? __ldcg(other(i) + (size_t)2 * TR * D + prow) : -INFINITY;
          ol[i] = in ? __ldcg(other(i) + (size_t)2 * TR * (D + 1) + prow) : -1.0f;
        }
#pragma unroll
        for (int i = 0; i < kOthers; ++i) top = fmaxf(top, om[i]);
        const float tb = top == -INFINITY ? 0.0f : top, of = ex2_approx(m - tb);
#pragma unroll
        for (int i = 0; i <= kOthers; ++i) {  // in order, this CTA's in its place
          if (own == i && cnt > 0) sum = fmaf(of, l, sum);
          if (i == kOthers) break;
          om[i] = ex2_approx(om[i] - tb);
          if (!(ol[i] < 0.0f)) sum = fmaf(om[i], ol[i], sum);
        }
        const float inv = normaliser(sum, at.r.kv - at.r.n + at.tok(sl) + tok);
        // 32 columns at a time, all their loads in flight at once
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          float4 v[kOthers][8];
#pragma unroll
          for (int i = 0; i < kOthers; ++i)
            if (!(ol[i] < 0.0f))
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[i][e] = __ldcg(reinterpret_cast<const float4*>(other(i)) + (size_t)(cc * 8 + e) * (2 * TR) + prow);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int col = cc * 32 + half * 16;
            uint32_t ov[16];
            if (cnt > 0) {
              tmem_ld_32x32b_x16(tmem_row(tmem, quarter, o_col + (uint32_t)col), ov);
              tmem_ld_wait();
              if (hurt) spoil(ov, col);
            }
            float acc[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
#pragma unroll
            for (int i = 0; i <= kOthers; ++i) {
              if (own == i && cnt > 0)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[e] = fmaf(of, __uint_as_float(ov[e]), acc[e]);
              if (i < kOthers && !(ol[i] < 0.0f))
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float4 x = v[i][half * 4 + e];
                  acc[4 * e] = fmaf(om[i], x.x, acc[4 * e]);
                  acc[4 * e + 1] = fmaf(om[i], x.y, acc[4 * e + 1]);
                  acc[4 * e + 2] = fmaf(om[i], x.z, acc[4 * e + 2]);
                  acc[4 * e + 3] = fmaf(om[i], x.w, acc[4 * e + 3]);
                }
            }
            if (live) store_row16(dst + col, acc, inv);
          }
        }
        if (live) put_lse(row, head, top, sum);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (warp < 4 || *c.abort_flag) return;
  // ---- split pieces left to be joined here: the last arrival at a group's
  // counter adds the group's parts, the last at the item's the groups', in
  // order and with the same operations as above; the elements of the live rows
  // are dealt to all row threads.
  const size_t pf = many_part_floats(D);
  float* const weights = reinterpret_cast<float*>(c.base_ptr);  // [top, sum, parts][row]: the tiles are done with
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!sh.join[which]) continue;
    // the first join ends without a barrier, and its slower warps still read the weights that this one replaces
    if (which && sh.join[0]) row_warps_meet();
    cur.b = sh.place[which][0];
    cur.h = sh.place[which][1];
    cur.k = sh.place[which][2];
    cur.nkv = sh.place[which][3];
    cur.u = sh.place[which][4];
    cur.j0 = 0;
    cur.r = many_request<WIN>(A, cur.b);
    const ManySplit split(cur, units, ctas);
    const int g = split.group();
    // the rows of the item that are any token's: slot 0's first live0, slot 1's first live1
    const int live0 = (cur.r.n - cur.tok(0) < cur.r.tt ? cur.r.n - cur.tok(0) : cur.r.tt) * A.group;
    const int live1 = !cur.two() ? 0 : (cur.r.n - cur.tok(1) < cur.r.tt ? cur.r.n - cur.tok(1) : cur.r.tt) * A.group;
    const int work = (live0 + live1) * (D / 16);
    bool of_groups = false;
#pragma unroll 1
    for (;;) {
      const bool final = of_groups || split.groups == 1;
      const int n = of_groups ? split.groups : split.members(g);
      const auto source = [&](int x) {
        return of_groups ? split.group_part(parts, pf, x) : split.part(parts, pf, g * split.gsize + x);
      };
      __threadfence();
      // the weights of each row's parts (-1: there is no O), its maximum and sum
      {
        const int prow = (int)threadIdx.x - 128;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
        for (int x = 0; x < n; ++x) top = fmaxf(top, __ldcg(source(x) + (size_t)2 * TR * D + prow));
        const float tb = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
        for (int x = 0; x < n; ++x) {
          const float pl = __ldcg(source(x) + (size_t)2 * TR * (D + 1) + prow);
          const float f = ex2_approx(__ldcg(source(x) + (size_t)2 * TR * D + prow) - tb);
          weights[(2 + x) * 2 * TR + prow] = pl < 0.0f ? -1.0f : f;
          if (!(pl < 0.0f)) sum = fmaf(f, pl, sum);
        }
        weights[prow] = top;
        weights[2 * TR + prow] = sum;
      }
      row_warps_meet();
      // 16 columns of a row to a thread (consecutive threads: rows), of four parts at a time
#pragma unroll 1
      for (int w = (int)threadIdx.x - 128; w < work; w += 256) {
        const int q = w % (live0 + live1), col4 = w / (live0 + live1) * 4;
        const int qs = q >= live0 ? 1 : 0, qr = q - (qs ? live0 : 0), prow = qs * TR + qr;
        float acc[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
#pragma unroll 1
        for (int x0 = 0; x0 < n; x0 += 4) {
          float f[4];
          float4 v[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] = x0 + i < n ? weights[(2 + x0 + i) * 2 * TR + prow] : -1.0f;
            if (f[i] == -1.0f) continue;
            const float* const from = source(x0 + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[i][e] = __ldcg(reinterpret_cast<const float4*>(from) + (size_t)(col4 + e) * (2 * TR) + prow);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (f[i] == -1.0f) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[4 * e] = fmaf(f[i], v[i][e].x, acc[4 * e]);
              acc[4 * e + 1] = fmaf(f[i], v[i][e].y, acc[4 * e + 1]);
              acc[4 * e + 2] = fmaf(f[i], v[i][e].z, acc[4 * e + 2]);
              acc[4 * e + 3] = fmaf(f[i], v[i][e].w, acc[4 * e + 3]);
            }
          }
        }
        const float top = weights[prow], sum = weights[2 * TR + prow];
        if (final) {
          const int tok = qr / A.group, head = cur.h * A.group + (qr - tok * A.group);
          const int64_t row = (int64_t)cur.r.q0 + cur.tok(qs) + tok;
          store_row16(A.o + row * A.o_token + (int64_t)head * A.o_head + col4 * 4, acc,
                      normaliser(sum, cur.r.kv - cur.r.n + cur.tok(qs) + tok));
          if (A.lse && col4 == 0)
            A.lse[row * (int64_t)(A.group * A.c.kv_heads) + head] =
                sum == 0.0f ? -INFINITY : ((top == -INFINITY ? 0.0f : top) + log2f(sum)) * kLn2;
        } else {
          float* const to = split.group_part(parts, pf, g);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            __stcg(reinterpret_cast<float4*>(to) + (size_t)(col4 + e) * (2 * TR) + prow,
                   make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]));
          if (col4 == 0) {
            __stcg(to + (size_t)2 * TR * D + prow, top);
            __stcg(to + (size_t)2 * TR * (D + 1) + prow, sum);
          }
        }
      }
      if (final) break;
      row_warps_meet();
      if (threadIdx.x == 128) {
        __threadfence();
        const unsigned n2 = (unsigned)split.groups;
        sh.last = atomicInc(counters + 2 * gridDim.x + split.c0, n2 - 1) == n2 - 1;
      }
      row_warps_meet();
      if (!*reinterpret_cast<volatile int*>(&sh.last)) break;
      of_groups = true;
    }
  }
}

constexpr int kManyCounters = 1024;  // of the context's counters; the kernel for few rows has the others but the last
constexpr int kWaitedWord = kPagedCounters - 1;

size_t few_workspace_floats(const tp3d_ctx* ctx, int d) {
  return (size_t)ctx->num_sms * FewShape<4>::kPerSm * kFewSlots * few_part_floats(d);
}

PFN_cuTensorMapEncodeTiled_v12000 encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// a bf16 array of `rank` dimensions (columns first, strides in elements), boxes of 64 columns with the 128-byte swizzle
tp3d_status row_map(CUtensorMap* m, const void* ptr, int rank, const int64_t* dims, const int64_t* strides,
                    const uint32_t* box) {
  auto fn = encode();
  if (!fn) return TP3D_ECUDA;
  cuuint64_t d[4], st[3];
  cuuint32_t bx[4], es[4];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    bx[i] = box[i];
    es[i] = 1;
    if (i > 0) {
      st[i - 1] = (cuuint64_t)strides[i - 1] * 2;
    }
  }
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), d, st, bx, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? TP3D_OK : TP3D_ECUDA;
}

// The kernels' shared-memory limits, set once per context (a context has one
// device), and the register split checked: setmaxnreg.inc waits until the
// block's launch registers cover it.
template <int D, bool WIN>
tp3d_status ready(tp3d_ctx* ctx) {
  const int bit = (D == 128 ? 1 : 2) << (WIN ? 4 : 0);
  if (ctx->paged_ready & bit) return TP3D_OK;
  TP3D_CUDA_TRY(cudaFuncSetAttribute(paged_attn_few_kernel<D, 4, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)few_smem<4>(D)));
  TP3D_CUDA_TRY(cudaFuncSetAttribute(paged_attn_few_kernel<D, 8, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)few_smem<8>(D)));
  TP3D_CUDA_TRY(cudaFuncSetAttribute(paged_attn_many_kernel<D, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kManySmem));
  cudaFuncAttributes fa;
  TP3D_CUDA_TRY(cudaFuncGetAttributes(&fa, paged_attn_many_kernel<D, WIN>));
  if (fa.numRegs * kManyThreads < 128 * kManyRegsLow + 256 * kManyRegsHigh) return TP3D_EUNSUPPORTED;
  ctx->paged_ready |= bit;
  return TP3D_OK;
}

// `after`: right after the other kernel of this call.  It then works beside
// that one, on the SMs that one leaves: the two write different rows, parts
// and counters, and it ends only when that one has ended.
template <int D, int W, bool WIN>
tp3d_status launch_few(tp3d_ctx* ctx, const PagedAttn& A, bool after, float* parts, cudaStream_t s) {
  return launch_dependent(paged_attn_few_kernel<D, W, WIN>, (unsigned)(ctx->num_sms * FewShape<W>::kPerSm),
                          FewShape<W>::kThreads, few_smem<W>(D), s, A, !after, parts, ctx->d_paged + kManyCounters,
                          ctx->d_paged + kWaitedWord);
}

template <int D, bool WIN>
tp3d_status launch_many(tp3d_ctx* ctx, const PagedAttn& A, bool few, float* parts, cudaStream_t s) {
  CUtensorMap mq, mk, mv;
  const int64_t qd[3] = {D, (int64_t)A.group * A.c.kv_heads, A.tokens}, qs[2] = {A.q_head, A.q_token};
  const uint32_t qb[3] = {64, (uint32_t)A.group, (uint32_t)(TR / A.group)};
  TP3D_TRY(row_map(&mq, A.q, 3, qd, qs, qb));
  const int64_t cd[4] = {D, A.c.page, A.c.kv_heads, A.c.pages};
  const int64_t cs[3] = {A.c.token_stride, A.c.head_stride, A.c.page_stride};
  const uint32_t cb[4] = {64, (uint32_t)(A.c.page < TR ? A.c.page : TR), 1, 1};
  TP3D_TRY(row_map(&mk, A.c.k, 4, cd, cs, cb));
  TP3D_TRY(row_map(&mv, A.c.v, 4, cd, cs, cb));
  return launch_dependent(paged_attn_many_kernel<D, WIN>, (unsigned)ctx->num_sms, kManyThreads, kManySmem, s, mq, mk,
                          mv, A, parts, ctx->d_paged, few ? ctx->d_paged + kWaitedWord : nullptr);
}

template <int D, bool WIN>
tp3d_status launch(tp3d_ctx* ctx, const PagedAttn& A, bool few, bool many, bool wide, void* workspace, cudaStream_t s) {
  float* const few_parts = static_cast<float*>(workspace);
  TP3D_TRY((ready<D, WIN>(ctx)));
  if (many) TP3D_TRY((launch_many<D, WIN>(ctx, A, few, few_parts + few_workspace_floats(ctx, D), s)));
  if (!few) return TP3D_OK;
  return wide ? launch_few<D, 8, WIN>(ctx, A, many, few_parts, s) : launch_few<D, 4, WIN>(ctx, A, many, few_parts, s);
}

// The most keys that the rows of a request see between them, or 0 where the
// window is as wide as the tables: that leaves nothing out and goes the way of
// the call without one, to the same results.
int64_t window_keys(const PagedAttn& A, int64_t most_new) {
  const int64_t keys = (int64_t)A.window + A.sinks + most_new;
  return A.window > 0 && keys < A.width * A.c.page ? keys : 0;
}

// Whether a windowed call is little enough work for the kernel for few rows to
// take all of its requests, whatever rows they have.  There each block of 16
// rows reads every key that its request's rows see (the other blocks' from L2),
// so its time grows with blocks x keys over the SMs; the other kernel has one
// read for 256 rows but begins later, and an item that it cuts into many parts
// costs it their join, more the fewer items there are.  The window bounds the
// keys of every request, so the host knows both.  Here | there, heads of 128, us:
//   1 item   64 rows 11.8 | 17.7 (window 1167), 512 14.7 | 32.6, 1024 26.6 | 38.0 (2048), 2048 61.2 | 45.3 (4096)
//   8 items  128 rows 18.7 | 23.4 (1167), 256 32.9 | 37.4 (2048), 256 50.1 | 43.5 (4096), 512 44.5 | 36.3 (1167)
//   16       64 rows 18.6 | 22.5 (1167), 128 25.2 | 26.5 (1167), 128 33.1 | 29.5 (2048), 192 17.3 | 15.6 (128)
//   32       64 rows 9.9 | 14.5 (128), 64 18.4 | 21.2 (512), 64 25.4 | 23.1 (1167)
// Rows far beyond one another's windows do not see most of those keys: 2048 rows of 512 tokens, window 128, 22.1 | 18.1.
bool short_window(const tp3d_ctx* ctx, const PagedAttn& A, int64_t most_new) {
  const int64_t items = (int64_t)A.requests * A.c.kv_heads, blocks = items * ((most_new * A.group + 15) / 16);
  const int64_t keys = window_keys(A, most_new);
  if (keys == 0 || most_new > 2 * (int64_t)A.window) return false;
  if (items <= 0 || blocks * 8 > ctx->num_sms * 7) return false;  // measured up to 128
  const int64_t per_sm = (1 << 14) / items;
  return blocks * keys <= ctx->num_sms * (per_sm < 2048 ? per_sm : 2048);
}

}  // namespace

size_t paged_attn_workspace(const tp3d_ctx* ctx, int d) {
  return (few_workspace_floats(ctx, d) + (size_t)ctx->num_sms * kManySlots * many_part_floats(d)) * sizeof(float);
}

tp3d_status launch_paged_attn(tp3d_ctx* ctx, PagedAttn& A, int max_new, void* workspace, cudaStream_t s) {
  if (ctx->num_sms * 3 > kManyCounters || kManyCounters + ctx->num_sms * FewShape<4>::kPerSm * 3 > kWaitedWord)
    return TP3D_EUNSUPPORTED;
  // items (requests x key/value heads) that leave half of the SMs without one: see FewShape
  const bool wide = (int64_t)A.requests * A.c.kv_heads * 2 <= ctx->num_sms;
  const int64_t most_new = max_new > 0 && max_new < A.tokens ? max_new : A.tokens, most = most_new * A.group;
  int few_rows = wide ? FewShape<8>::kRows : FewShape<4>::kRows;
  if (short_window(ctx, A, most_new))
    few_rows = most > few_rows ? (int)most : few_rows;
  else if (!wide && window_keys(A, most_new) > 0 &&
           (A.c.head_dim == 64 || (int64_t)A.window + A.sinks <= FewShape<4>::kKeysWindow))
    few_rows = FewShape<4>::kRowsWindow;
  const bool many = most > few_rows;
  // One request that may have many rows goes to that kernel whatever it has
  // (all its rows are computed there all the same, and a launch is saved).
  const bool few = !many || A.requests > 1;
  A.few_rows = few ? few_rows : 0;
  if (A.window > 0)
    return A.c.head_dim == 128 ? launch<128, true>(ctx, A, few, many, wide, workspace, s)
                               : launch<64, true>(ctx, A, few, many, wide, workspace, s);
  return A.c.head_dim == 128 ? launch<128, false>(ctx, A, few, many, wide, workspace, s)
                             : launch<64, false>(ctx, A, few, many, wide, workspace, s);
}

}  // namespace tp3d
