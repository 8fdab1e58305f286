// paged_pages.cu - sharing, giving back and moving the pages of the paged
// key/value cache: tp3d_paged_fork, tp3d_paged_free, tp3d_paged_compact and
// tp3d_paged_copy of include/tp3d_paged.h.
//
// The bookkeeping moves a few words per table entry and per page, so launches
// and dependent reads bound it.  Entries are dealt evenly to all threads whatever
// the rows' lengths: every CTA forms the exclusive sums of the rows' entries in
// shared memory (16384 rows at most) and a thread finds its entry's row by a
// search in them, as in the plan.  Lists of pages come out in the order of the
// page numbers, whatever the order in which threads come: pages are counted by
// chunk while they are marked, and a second kernel, chunk by chunk, ranks them.
// The marks lie in the share counts, the chunks' counts in words of the context
// that are zero between calls.
//
// On the GPU, in a captured graph: 448 forks of 64 requests of up to 8000 tokens
// in pages of 16 (112000 entries) 5.3 us, 31000 pages given back 8.9 us in two
// launches, a pool of 9233 pages compacted 9.1 us in three, without the copies.  A
// call from Python takes 4 to 7 us of the host.
#include <initializer_list>

#include "paged.cuh"

namespace tp3d {

namespace {

constexpr int kMaxRows = 16384;
constexpr int kChunks = 1024;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
// Counts by chunk, several of each, so that the CTAs' additions do not all meet in
// a few lines of L2 (31000 pages given back in 152 chunks: 8.9 us, with one of each
// 14.6).
constexpr int kCopies = 8;
// in the context's words: the counts (a compaction has two kinds), arrivals, whether the free list is bad (zero
// between calls), and that again (each call writes it before it is read)
constexpr int kCounts = kPageWords, kArrivals = kCounts + 2 * kCopies * kChunks, kBad = kArrivals + 1, kWasBad = kBad + 1;
static_assert(kWasBad < kPagedWords, "the context's words");
// the word to count a page of a chunk in
__device__ __forceinline__ unsigned* count_word(unsigned* words, int kind, int64_t chunk) {
  return words + kCounts + (kind * kCopies + (blockIdx.x & (kCopies - 1))) * kChunks + chunk;
}
__device__ __forceinline__ long long count_of(const unsigned* words, int kind, int chunk) {
  unsigned n = 0;
#pragma unroll
  for (int i = 0; i < kCopies; ++i) n += ld_plain(words + kCounts + (kind * kCopies + i) * kChunks + chunk);
  return n;
}

struct Pool {
  int page_log2, rows, chunk_log2;
  int64_t pages, width, free_cap;
  int32_t *table, *shares, *free_pages;
  unsigned* words;
  int* err;
};

// The sums over the threads before this one of x, and (total) over all.
__device__ __forceinline__ long long block_scan(long long x, long long (&warp_sum)[kWarps], long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) warp_sum[warp] = y;
  __syncthreads();
  y -= x;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) y += warp_sum[w];
    total += warp_sum[w];
  }
  return y;
}

// sums[i] = the sum of entries(j) over j < i, for i < n; returns that over all.
// Whoever reads them synchronises first.
template <class F>
__device__ __forceinline__ long long sum_rows(int n, int32_t* sums, const F& entries) {
  __shared__ long long warp_sum[kWarps];
  long long carry = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + (int)threadIdx.x;
    long long total;
    const long long at = carry + block_scan(i < n ? entries(i) : 0, warp_sum, total);
    if (i < n) sums[i] = (int32_t)(at < INT32_MAX ? at : INT32_MAX);
    carry += total;
  }
  return carry;
}

__device__ __forceinline__ int64_t clamp_count(const int32_t* count, int64_t cap) {
  const int64_t n = ld_plain(count);
  return n < 0 ? 0 : n > cap ? cap : n;
}

// ------------------------------------------------------------------ fork
struct ForkArgs {
  Pool P;
  int forks;
  const int32_t *src, *dst, *len, *free_count;
  int32_t *free_left, *copy_from, *copy_to, *copy_count;
};

// Every CTA looks all forks and the free pages that they take over first, so all
// of them come to the same answer before any writes: a fork reads rows that are no
// fork's target.  (Entries of whole pages are read once, as they are copied: one past
// the pool becomes -1 there.)
__global__ void __launch_bounds__(kThreads) paged_fork_kernel(const ForkArgs F) {
  extern __shared__ int32_t smem[];
  __shared__ long long warp_sum[kWarps];
  int32_t* const cols = smem;             // exclusive sums of the entries
  int32_t* const parts = smem + F.forks;  // exclusive sums of the partly filled pages
  uint32_t* const is_src = reinterpret_cast<uint32_t*>(smem + 2 * F.forks);
  const int row_words = (F.P.rows + 31) / 32;
  uint32_t* const is_dst = is_src + row_words;
  const int64_t cap = F.P.width << F.P.page_log2;
  const int in_page = (1 << F.P.page_log2) - 1;
  for (int i = threadIdx.x; i < 2 * row_words; i += kThreads) is_src[i] = 0;
  grid_begin();
  __syncthreads();
  const int64_t count0 = ld_plain(F.free_count), count = clamp_count(F.free_count, F.P.free_cap);
  bool bad = count != count0;
  int bad_page = INT32_MAX;  // the first place from the list's top, of this thread's, whose entry is no page
  long long carry = 0;       // both sums: 2^41 entries at most below, partly filled pages above
  constexpr int kPart = 46;
  for (int base = 0; base < F.forks; base += kThreads) {
    const int i = base + (int)threadIdx.x;
    long long mine = 0, total;
    int32_t e = 0, page = 0;
    if (i < F.forks) {
      const int s = ld_plain(F.src + i), d = ld_plain(F.dst + i), len = ld_plain(F.len + i);
      // a place of the list's top for each fork, which takes one or none
      page = i < count ? ld_plain(F.P.free_pages + (count - 1 - i)) : 0;
      if (s >= 0 && s < F.P.rows && d >= 0 && d < F.P.rows && len >= 0 && len <= cap && len <= kPagedMaxTokens) {
        mine = pages_of(len, F.P.page_log2);
        if (len & in_page) {
          e = ld_plain(F.P.table + s * F.P.width + (len >> F.P.page_log2));
          mine += 1LL << kPart;
        }
        atomicOr(is_src + (s >> 5), 1u << (s & 31));
        bad |= (atomicOr(is_dst + (d >> 5), 1u << (d & 31)) >> (d & 31)) & 1u;
      } else {
        bad = true;
      }
    }
    const long long at = carry + block_scan(mine, warp_sum, total);
    // (looked at behind the sums, which do not wait for them: 448 forks 5.3 us, before them 6.6)
    bad |= e < 0 || e >= F.P.pages;
    if ((page < 0 || page >= F.P.pages) && i < bad_page) bad_page = i;
    if (i < F.forks) {
      const long long n = at & ((1LL << kPart) - 1);
      cols[i] = (int32_t)(n < INT32_MAX ? n : INT32_MAX);
      parts[i] = (int32_t)(at >> kPart);
    }
    carry += total;
  }
  const long long entries = carry & ((1LL << kPart) - 1), fresh = carry >> kPart;
  __syncthreads();
  for (int i = threadIdx.x; i < row_words; i += kThreads) bad |= (is_src[i] & is_dst[i]) != 0;
  bad |= bad_page < fresh || fresh > count || entries > INT32_MAX;
  bad = __syncthreads_or(bad);  // (and the sums are in)
  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
  if (tid == 0) {
    if (bad) raise_error(F.P.err, TP3D_EPAGES);
    *F.copy_count = bad ? 0 : (int32_t)fresh;
    *F.free_left = (int32_t)(bad ? count : count - fresh);
  }
  if (bad) return;
  for (int64_t x = tid; x < entries; x += step) {
    const int i = last_at_most(cols, F.forks, (int32_t)x);
    const int s = ld_plain(F.src + i), d = ld_plain(F.dst + i), len = ld_plain(F.len + i);
    const int64_t col = x - cols[i];
    int32_t e = ld_plain(F.P.table + s * F.P.width + col);
    if (col < len >> F.P.page_log2) {
      if (e >= F.P.pages) {
        raise_error(F.P.err, TP3D_EPAGES);
        e = -1;
      }
      if (e >= 0) atomicAdd(F.P.shares + e, 1);
    } else {
      const int n = parts[i];
      const int32_t page = ld_plain(F.P.free_pages + (count - 1 - n));
      F.copy_from[n] = e;
      F.copy_to[n] = page;
      e = page;
    }
    F.P.table[d * F.P.width + col] = e;
  }
}

// ------------------------------------------------------------------ free
struct FreeArgs {
  Pool P;
  const int32_t *first, *end, *free_count;
  int32_t* free_left;
};
// A page whose last owner is gone: so much is taken from its shares, which no
// number of owners given up too many brings back.
constexpr int kGone = 1 << 30;

__global__ void __launch_bounds__(kThreads) paged_free_mark_kernel(const FreeArgs F) {
  extern __shared__ int32_t smem[];
  grid_begin();
  bool bad = false;
  const long long entries = sum_rows(F.P.rows, smem, [&](int r) -> long long {
    const int32_t a = ld_plain(F.first + r), b = ld_plain(F.end + r);
    if (b <= a) return 0;
    const bool out = a < 0 || b > F.P.width;
    bad |= out;
    return out ? 0 : b - a;
  });
  if (entries > INT32_MAX) bad = true;
  if (bad) raise_error(F.P.err, TP3D_EPAGES);
  __syncthreads();
  if (entries > INT32_MAX) return;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x; x < entries; x += step) {
    const int r = last_at_most(smem, F.P.rows, (int32_t)x);
    int32_t* const at = F.P.table + r * F.P.width + ld_plain(F.first + r) + (x - smem[r]);
    const int32_t e = *at;
    if (e < 0) continue;
    *at = -1;
    if (e >= F.P.pages) {
      raise_error(F.P.err, TP3D_EPAGES);
      continue;
    }
    const int old = atomicSub(F.P.shares + e, 1);
    if (old == 0) {
      atomicSub(F.P.shares + e, kGone);
      atomicAdd(count_word(F.P.words, 0, e >> F.P.chunk_log2), 1u);
    } else if (old < 0) {
      raise_error(F.P.err, TP3D_EPAGES);
    }
  }
}

__global__ void __launch_bounds__(kThreads) paged_free_list_kernel(const FreeArgs F) {
  __shared__ int32_t above[kChunks];  // pages freed in the chunks from the last one down to this, less its own
  __shared__ long long warp_sum[kWarps];
  __shared__ int last;
  grid_begin();
  const int chunks = (int)((F.P.pages + (1LL << F.P.chunk_log2) - 1) >> F.P.chunk_log2);
  const int64_t size = 1LL << F.P.chunk_log2;
  const auto page = [&](int i, int64_t base) { return ((int64_t)(chunks - 1 - i) << F.P.chunk_log2) + base - 1 - threadIdx.x; };
  const auto share = [&](int64_t p) { return p < F.P.pages ? ld_plain(F.P.shares + p) : 0; };
  int32_t first = share(page(blockIdx.x, size));  // on its way while the counts are added up
  const long long freed = sum_rows(chunks, above, [&](int i) { return count_of(F.P.words, 0, chunks - 1 - i); });
  __syncthreads();
  const int64_t count0 = ld_plain(F.free_count), count = clamp_count(F.free_count, F.P.free_cap);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const int64_t left = count + freed;
    if (count != count0 || left > F.P.free_cap) raise_error(F.P.err, TP3D_EPAGES);
    *F.free_left = (int32_t)(left < F.P.free_cap ? left : F.P.free_cap);
  }
  for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
    int64_t at = count + above[i];
    if ((i + 1 < chunks ? above[i + 1] : freed) == above[i]) continue;
    for (int64_t base = size; base > 0; base -= kThreads) {
      const int64_t p = page(i, base);
      const bool gone = (i == blockIdx.x && base == size ? first : share(p)) < -kGone / 2;
      long long total;
      const int64_t to = at + block_scan(gone, warp_sum, total);
      at += total;
      if (!gone) continue;
      F.P.shares[p] = 0;
      if (to < F.P.free_cap) F.P.free_pages[to] = (int32_t)p;
    }
  }
  // the last CTA to come, when all have read the counts, clears them
  __syncthreads();
  if (threadIdx.x == 0) last = arrive_last(F.P.words + kArrivals, gridDim.x);
  __syncthreads();
  if (last)
    for (int k = 0; k < kCopies; ++k)
      for (int i = threadIdx.x; i < chunks; i += kThreads) F.P.words[kCounts + k * kChunks + i] = 0;
}

// ------------------------------------------------------------------ compact
struct CompactArgs {
  Pool P;
  const int32_t *kv_len, *free_count;
  int32_t *map, *copy_from, *copy_to, *copy_count;
};
constexpr int kIsFree = INT32_MIN;  // the share count of a page that the free list names

__device__ __forceinline__ bool good_count(const CompactArgs& C, int64_t& count) {
  count = ld_plain(C.free_count);
  return count >= 0 && count <= C.P.pages;
}

// Marks the free pages, and counts them by chunk: those below `used` (the places
// to fill), and the others.
__global__ void __launch_bounds__(kThreads) paged_compact_mark_kernel(const CompactArgs C) {
  grid_begin();
  int64_t count;
  bool bad = !good_count(C, count);
  const int64_t used = C.P.pages - count, step = (int64_t)gridDim.x * kThreads;
  if (!bad)
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < count; i += step) {
      const int32_t p = ld_plain(C.P.free_pages + i);
      if (p < 0 || p >= C.P.pages || atomicExch(C.P.shares + p, kIsFree) == kIsFree) {
        bad = true;
        continue;
      }
      atomicAdd(count_word(C.P.words, p < used ? 0 : 1, p >> C.P.chunk_log2), 1u);
    }
  if (bad) {
    raise_error(C.P.err, TP3D_EPAGES);
    C.P.words[kBad] = 1;
  }
}

// The two lists, and the map; a page that moves has -2 - n there, for its place n in the lists.
__global__ void __launch_bounds__(kThreads) paged_compact_list_kernel(const CompactArgs C) {
  __shared__ int32_t holes[kChunks], movers[kChunks];
  __shared__ long long warp_sum[kWarps];
  grid_begin();
  int64_t count;
  good_count(C, count);
  const int64_t used = C.P.pages - count, size = 1LL << C.P.chunk_log2;
  const auto share = [&](int64_t p) { return p < C.P.pages ? ld_plain(C.P.shares + p) : 0; };
  const int32_t ahead = share(blockIdx.x * size + threadIdx.x);  // on its way while the counts are added up
  const bool bad = C.P.words[kBad] != 0;
  const int chunks = (int)((C.P.pages + size - 1) >> C.P.chunk_log2);
  long long carry = 0;  // both sums: places to fill below, pages that move above
  for (int base = 0; base < chunks; base += kThreads) {
    const int i = base + (int)threadIdx.x;
    long long mine = 0, total;
    if (i < chunks) {
      const int64_t lo = i * size > used ? i * size : used, hi = (i + 1) * size < C.P.pages ? (i + 1) * size : C.P.pages;
      mine = count_of(C.P.words, 0, i) + ((hi > lo ? hi - lo - count_of(C.P.words, 1, i) : 0) << 32);
    }
    const long long at = carry + block_scan(mine, warp_sum, total);
    if (i < chunks) {
      holes[i] = (int32_t)(at & 0xffffffffLL);
      movers[i] = (int32_t)(at >> 32);
    }
    carry += total;
  }
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *C.copy_count = bad ? 0 : (int32_t)(carry & 0xffffffffLL);
    C.P.words[kWasBad] = bad;
  }
  const int64_t most = C.P.pages / 2;
  for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
    int64_t hole_at = holes[i], mover_at = movers[i];
    for (int64_t base = 0; base < size; base += kThreads) {
      const int64_t p = i * size + base + threadIdx.x;
      if (i * size + base >= C.P.pages) break;
      const bool in = p < C.P.pages, free = (i == blockIdx.x && base == 0 ? ahead : share(p)) == kIsFree;
      const bool hole = free && p < used, mover = in && !free && p >= used;
      long long total;  // both ranks in one sum
      const long long at = block_scan((hole ? 1LL : 0) + (mover ? 1LL << 32 : 0), warp_sum, total);
      const int64_t h = hole_at + (at & 0xffffffffLL), m = mover_at + (at >> 32);
      hole_at += total & 0xffffffffLL;
      mover_at += total >> 32;
      if (free) C.P.shares[p] = 0;
      if (bad) {
        if (in) C.map[p] = (int32_t)p;
        continue;
      }
      if (hole && h < most) C.copy_to[h] = (int32_t)p;
      if (mover && m < most) C.copy_from[m] = (int32_t)p;
      if (in) C.map[p] = mover ? (int32_t)(-2 - m) : free ? -1 : (int32_t)p;
    }
  }
}

// Shares, map and free list follow the moves, and the tables' entries.  An entry's
// reader finds a moved page's word in the map as it was or already with the new
// page, and comes to the same page by either (relaxed accesses, both of 32 bits).
__global__ void __launch_bounds__(kThreads) paged_compact_move_kernel(const CompactArgs C) {
  extern __shared__ int32_t smem[];
  grid_begin();
  const bool bad = C.P.words[kWasBad] != 0;
  int64_t count;
  good_count(C, count);
  const int64_t cap = C.P.width << C.P.page_log2;
  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
  // what the two kernels before this have read is zero again
  for (int64_t i = tid; i < 2 * kCopies * kChunks; i += step) C.P.words[kCounts + i] = 0;
  if (tid == 0) C.P.words[kBad] = 0;
  if (!bad) {
    const int32_t moves = ld_plain(C.copy_count);
    for (int64_t i = tid; i < moves; i += step) {
      const int32_t from = ld_plain(C.copy_from + i), to = ld_plain(C.copy_to + i);
      asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(C.map + from), "r"(to) : "memory");
      C.P.shares[to] = ld_plain(C.P.shares + from);
      C.P.shares[from] = 0;
    }
    for (int64_t i = tid; i < count; i += step) C.P.free_pages[i] = (int32_t)(C.P.pages - 1 - i);
    bool wrong = false;
    const long long entries = sum_rows(C.P.rows, smem, [&](int r) -> long long {
      const int32_t kv = ld_plain(C.kv_len + r);
      const bool fits = kv >= 0 && kv <= cap && kv <= kPagedMaxTokens;
      wrong |= !fits;
      return fits ? pages_of(kv, C.P.page_log2) : 0;
    });
    __syncthreads();
    for (int64_t x = tid; x < entries && entries <= INT32_MAX; x += step) {
      const int r = last_at_most(smem, C.P.rows, (int32_t)x);
      int32_t* const at = C.P.table + r * C.P.width + (x - smem[r]);
      const int32_t e = *at;
      if (e < 0) continue;
      int32_t now = -1;
      if (e < C.P.pages) asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(now) : "l"(C.map + e) : "memory");
      if (now < -1) now = -2 - now < moves ? ld_plain(C.copy_to + (-2 - now)) : -1;
      if (now < 0) wrong = true;
      else if (now != e) *at = now;
    }
    if (wrong || entries > INT32_MAX) raise_error(C.P.err, TP3D_EPAGES);
  }
}

// ------------------------------------------------------------------ copy
// 16-byte vectors of a page, from the innermost: `run` contiguous ones, n1 runs
// s1 vectors apart, and whatever is left s2 apart (host side: longest run).
struct CopyArgs {
  uint4 *k, *v;
  int64_t pages, page_stride;  // in vectors
  uint32_t vectors, run, n1;   // of a page: all; of a run; runs
  int64_t s1, s2;
  int64_t copies;
  const int32_t *from, *to, *count;
  int* err;
};
// Many more CTAs than there is room for, a tile or a few each: they come and go
// by themselves, which keeps reads and writes mixed (2333 pages of 64 KiB in K and
// V: 92 us, 0.97 of the copy rate; in a grid of four to an SM 103, of eight 94).
constexpr int kCopyThreads = 256, kCopyPerSm = 64;
constexpr int kCopyVecs = 8;                                          // in flight per thread
constexpr uint32_t kCopyTile = (uint32_t)kCopyThreads * kCopyVecs;  // 32 KiB

template <bool WHOLE>
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const CopyArgs C) {
  grid_begin();
  int64_t n = C.copies;
  if (C.count) {
    const int64_t count = ld_plain(C.count);
    if ((count < 0 || count > n) && blockIdx.x == 0 && threadIdx.x == 0) raise_error(C.err, TP3D_EPAGES);
    n = count < 0 ? 0 : count < n ? count : n;
  }
  const uint32_t tiles = (C.vectors + kCopyTile - 1) / kCopyTile;  // of a page and pool
  const int64_t all = n * 2 * tiles;
  for (int64_t x = blockIdx.x; x < all; x += gridDim.x) {
    // 32-bit division where it fits (as in the store)
    const int64_t pair = x >> 32 ? x / tiles : (int64_t)((uint32_t)x / tiles);
    const uint32_t v0 = (uint32_t)(x - pair * tiles) * kCopyTile + threadIdx.x;
    const int32_t from = ld_plain(C.from + (pair >> 1)), to = ld_plain(C.to + (pair >> 1));
    if (from < 0 || from >= C.pages || to < 0 || to >= C.pages) {
      if (threadIdx.x == 0) raise_error(C.err, TP3D_EPAGES);
      continue;
    }
    uint4* const pool = pair & 1 ? C.v : C.k;
    const uint4* const src = pool + from * C.page_stride;
    uint4* const dst = pool + to * C.page_stride;
    uint4 r[kCopyVecs];
    int64_t at[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      const uint32_t v = v0 + i * kCopyThreads;
      at[i] = v;
      if (!WHOLE) {
        const uint32_t k = v / C.run, o = k / C.n1;
        at[i] = (v - k * C.run) + (k - o * C.n1) * C.s1 + o * C.s2;
      }
      if (v < C.vectors) r[i] = ld_plain(src + at[i]);
    }
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (v0 + i * kCopyThreads < C.vectors) dst[at[i]] = r[i];
  }
}

// ------------------------------------------------------------------ host side
tp3d_status check_pool(const tp3d_ctx* ctx, const tp3d_page_pool* p, Pool* out) {
  if (!ctx || !p || p->rows < 0 || p->pages < 1 || p->table_width < 0 || p->free_cap < 0) return TP3D_EINVAL;
  if (!p->shares || !p->free_pages || (p->rows > 0 && p->table_width > 0 && !p->block_table)) return TP3D_EINVAL;
  const int pl = page_log2(p->page);
  if (pl < 0 || p->rows > kMaxRows || p->pages > INT32_MAX || p->table_width > INT32_MAX || p->free_cap > INT32_MAX)
    return TP3D_EUNSUPPORTED;
  if (p->free_cap < p->pages) return TP3D_ESHAPE;
  for (const void* x : {p->block_table, p->shares, p->free_pages})
    if (!aligned(x, 4)) return TP3D_EALIGN;
  int chunk = 9;  // a pass of a CTA at least
  while ((p->pages + (1LL << chunk) - 1) >> chunk > kChunks) ++chunk;
  *out = Pool{pl, p->rows, chunk, p->pages, p->table_width, p->free_cap, p->block_table, p->shares, p->free_pages,
              ctx->d_paged, ctx->d_err};
  return TP3D_OK;
}
size_t table_bytes(const Pool& P) { return (size_t)P.rows * P.width * 4; }

tp3d_status check_words(std::initializer_list<const void*> words) {
  for (const void* p : words)
    if (!p) return TP3D_EINVAL;
  for (const void* p : words)
    if (!aligned(p, 4)) return TP3D_EALIGN;
  return TP3D_OK;
}

// The kernels whose sums may pass 48 KiB get their largest size once per context.
constexpr int kPagesReady = 8;  // of tp3d_ctx::paged_ready
constexpr int kRowsSmem = kMaxRows * 4, kForkSmem = kMaxRows * 8 + kMaxRows / 4;
tp3d_status ready(tp3d_ctx* ctx) {
  if (ctx->paged_ready & kPagesReady) return TP3D_OK;
  TP3D_CUDA_TRY(cudaFuncSetAttribute(paged_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kForkSmem));
  TP3D_CUDA_TRY(cudaFuncSetAttribute(paged_free_mark_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem));
  TP3D_CUDA_TRY(cudaFuncSetAttribute(paged_compact_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem));
  ctx->paged_ready |= kPagesReady;
  return TP3D_OK;
}

unsigned grid_of(const tp3d_ctx* ctx, int64_t threads, size_t smem) {
  const int64_t n = (threads + kThreads - 1) / kThreads, most = (int64_t)ctx->num_sms * (smem > 48 * 1024 ? 1 : 2);
  return (unsigned)(n < 1 ? 1 : n < most ? n : most);
}
unsigned chunk_grid(const tp3d_ctx* ctx, const Pool& P) {
  const int64_t chunks = (P.pages + (1LL << P.chunk_log2) - 1) >> P.chunk_log2, most = (int64_t)ctx->num_sms * 2;
  return (unsigned)(chunks < most ? chunks : most);
}

}  // namespace

}  // namespace tp3d

using namespace tp3d;

extern "C" {

tp3d_status tp3d_paged_fork(tp3d_ctx* ctx, const tp3d_page_pool* pool, int forks, const int32_t* src,
                            const int32_t* dst, const int32_t* len, const int32_t* free_count, int32_t* free_left,
                            int32_t* copy_from, int32_t* copy_to, int32_t* copy_count, void* stream) {
  Pool P;
  TP3D_TRY(check_pool(ctx, pool, &P));
  if (forks < 0) return TP3D_EINVAL;
  if (forks > kMaxRows) return TP3D_EUNSUPPORTED;
  TP3D_TRY(check_words({free_count, free_left, copy_count}));
  if (forks > 0) TP3D_TRY(check_words({src, dst, len, copy_from, copy_to}));
  const size_t fb = (size_t)forks * 4;
  const Range out[] = {{P.table, table_bytes(P)}, {P.shares, (size_t)P.pages * 4}, {free_left, 4}, {copy_from, fb},
                       {copy_to, fb}, {copy_count, 4}};
  const Range in[] = {{src, fb}, {dst, fb}, {len, fb}, {P.free_pages, (size_t)P.free_cap * 4}, {free_count, 4}};
  if (clash(out, in)) return TP3D_EOVERLAP;
  TP3D_TRY(ready(ctx));
  const ForkArgs F{P, forks, src, dst, len, free_count, free_left, copy_from, copy_to, copy_count};
  const size_t smem = (size_t)forks * 8 + (size_t)((P.rows + 31) / 32) * 8;
  return launch_dependent(paged_fork_kernel, grid_of(ctx, forks * P.width, smem), kThreads, smem, as_stream(stream), F);
}

tp3d_status tp3d_paged_free(tp3d_ctx* ctx, const tp3d_page_pool* pool, const int32_t* first, const int32_t* end,
                            const int32_t* free_count, int32_t* free_left, void* stream) {
  Pool P;
  TP3D_TRY(check_pool(ctx, pool, &P));
  TP3D_TRY(check_words({free_count, free_left}));
  if (P.rows > 0) TP3D_TRY(check_words({first, end}));
  const size_t rb = (size_t)P.rows * 4;
  const Range out[] = {{P.table, table_bytes(P)}, {P.shares, (size_t)P.pages * 4},
                       {P.free_pages, (size_t)P.free_cap * 4}, {free_left, 4}};
  const Range in[] = {{first, rb}, {end, rb}, {free_count, 4}};
  if (clash(out, in)) return TP3D_EOVERLAP;
  TP3D_TRY(ready(ctx));
  const FreeArgs F{P, first, end, free_count, free_left};
  const cudaStream_t s = as_stream(stream);
  TP3D_TRY(launch_dependent(paged_free_mark_kernel, grid_of(ctx, P.rows * P.width, rb), kThreads, rb, s, F));
  return launch_dependent(paged_free_list_kernel, chunk_grid(ctx, P), kThreads, 0, s, F);
}

tp3d_status tp3d_paged_compact(tp3d_ctx* ctx, const tp3d_page_pool* pool, const int32_t* kv_len,
                               const int32_t* free_count, int32_t* page_map, int32_t* copy_from, int32_t* copy_to,
                               int32_t* copy_count, void* stream) {
  Pool P;
  TP3D_TRY(check_pool(ctx, pool, &P));
  TP3D_TRY(check_words({free_count, page_map, copy_count}));
  if (P.rows > 0) TP3D_TRY(check_words({kv_len}));
  if (P.pages > 1) TP3D_TRY(check_words({copy_from, copy_to}));
  const size_t rb = (size_t)P.rows * 4, pb = (size_t)P.pages * 4, cb = (size_t)(P.pages / 2) * 4;
  const Range out[] = {{P.table, table_bytes(P)}, {P.shares, pb}, {P.free_pages, (size_t)P.free_cap * 4},
                       {page_map, pb}, {copy_from, cb}, {copy_to, cb}, {copy_count, 4}};
  const Range in[] = {{kv_len, rb}, {free_count, 4}};
  if (clash(out, in)) return TP3D_EOVERLAP;
  TP3D_TRY(ready(ctx));
  const CompactArgs C{P, kv_len, free_count, page_map, copy_from, copy_to, copy_count};
  const cudaStream_t s = as_stream(stream);
  TP3D_TRY(launch_dependent(paged_compact_mark_kernel, grid_of(ctx, P.pages, 0), kThreads, 0, s, C));
  TP3D_TRY(launch_dependent(paged_compact_list_kernel, chunk_grid(ctx, P), kThreads, 0, s, C));
  const int64_t entries = P.rows * P.width;
  return launch_dependent(paged_compact_move_kernel, grid_of(ctx, entries > P.pages ? entries : P.pages, rb),
                          kThreads, rb, s, C);
}

tp3d_status tp3d_paged_copy(tp3d_ctx* ctx, const tp3d_kv_cache* cache, int64_t copies, const int32_t* copy_from,
                            const int32_t* copy_to, const int32_t* copy_count, void* stream) {
  if (!ctx || copies < 0) return TP3D_EINVAL;
  TP3D_TRY(check_cache(cache));
  if (copies > INT32_MAX) return TP3D_EUNSUPPORTED;
  if (copies == 0) return TP3D_OK;
  TP3D_TRY(check_words({copy_from, copy_to}));
  if (!aligned(copy_count, 4)) return TP3D_EALIGN;
  const size_t cb = cache_bytes(*cache);
  for (const void* pool : {cache->k, cache->v})
    if (overlaps(pool, cb, copy_from, (size_t)copies * 4) || overlaps(pool, cb, copy_to, (size_t)copies * 4) ||
        overlaps(pool, cb, copy_count, 4))
      return TP3D_EOVERLAP;
  // the dimension of the smaller stride inside
  const bool heads_in = cache->head_stride <= cache->token_stride;
  int64_t run = cache->head_dim / 8, n1 = heads_in ? cache->kv_heads : cache->page;
  int64_t n2 = heads_in ? cache->page : cache->kv_heads;
  int64_t s1 = (heads_in ? cache->head_stride : cache->token_stride) / 8;
  int64_t s2 = (heads_in ? cache->token_stride : cache->head_stride) / 8;
  if (s1 == run || n1 == 1) {  // rows without gaps are one run
    run *= n1;
    n1 = n2;
    s1 = s2;
    n2 = 1;
  }
  if (n2 == 1 && (s1 == run || n1 == 1)) {
    run *= n1;
    n1 = 1;
  }
  if (run * n1 * n2 > INT32_MAX) return TP3D_EUNSUPPORTED;
  CopyArgs C{};
  C.k = static_cast<uint4*>(cache->k);
  C.v = static_cast<uint4*>(cache->v);
  C.pages = cache->pages;
  C.page_stride = cache->page_stride / 8;
  C.vectors = (uint32_t)(run * n1 * n2);
  C.run = (uint32_t)run;
  C.n1 = (uint32_t)n1;
  C.s1 = s1;
  C.s2 = s2;
  C.copies = copies;
  C.from = copy_from;
  C.to = copy_to;
  C.count = copy_count;
  C.err = ctx->d_err;
  const int64_t tiles = copies * 2 * ((C.vectors + kCopyTile - 1) / kCopyTile), most = (int64_t)ctx->num_sms * kCopyPerSm;
  const unsigned grid = (unsigned)(tiles < most ? tiles : most);
  return n1 == 1 && n2 == 1 ? launch_dependent(paged_copy_kernel<true>, grid, kCopyThreads, 0, as_stream(stream), C)
                            : launch_dependent(paged_copy_kernel<false>, grid, kCopyThreads, 0, as_stream(stream), C);
}

}  // extern "C"
