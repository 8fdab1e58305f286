// attn_tile.cuh - what the tcgen05 attention kernels share: the shared-memory
// frame of 128-row tiles, operand descriptors, warp-level waits, and the
// 32-column row store.
#pragma once

#include "common.cuh"

namespace tp3d {

using bf16 = __nv_bfloat16;

constexpr int TR = 128;              // rows of a tile (queries or keys)
constexpr uint32_t kChunk = 16384;   // 128 rows x 64 bf16 columns (one 128-byte swizzle span)
constexpr uint32_t kTile = 2 * kChunk;  // a 128 x 128 bf16 tile
constexpr int kSmem = 7 * kTile + 512 + 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

#if defined(__CUDACC__)

struct Ctx {
  uint32_t base;       // 1024-aligned shared address of the tile area
  uint8_t* base_ptr;
  uint32_t bar0;       // first mbarrier
  volatile int* abort_flag;
  uint32_t* tmem_holder;
};

__device__ __forceinline__ Ctx setup_smem(uint8_t* smem_raw) {
  Ctx c;
  const uint32_t raw = smem_u32(smem_raw);
  c.base = (raw + 1023u) & ~1023u;
  c.base_ptr = smem_raw + (c.base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(c.base_ptr + 7 * kTile);
  c.bar0 = smem_u32(bars);
  c.tmem_holder = reinterpret_cast<uint32_t*>(bars + 40);
  c.abort_flag = reinterpret_cast<volatile int*>(c.tmem_holder + 1);
  return c;
}

// descriptors of a 128-row tile stored as 64-column swizzled chunks
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t tile, int k16) {  // contraction along the columns
  return smem_desc_sw128(tile + (uint32_t)(k16 >> 2) * kChunk + (uint32_t)(k16 & 3) * 32u, 16u, 1024u);
}
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t tile, int k16) {  // contraction along the rows
  return smem_desc_sw128(tile + (uint32_t)k16 * 2048u, kChunk, 1024u);
}

__device__ __forceinline__ uint4 pack8f(const float* f) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return v;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Ctx& c, int* err, int lane) {
  bool ok = lane == 0 ? mbar_wait(bar, parity, c.abort_flag, err) : false;
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ uint32_t tmem_row(uint32_t tmem, int quarter, uint32_t col) {
  return tmem + ((uint32_t)(quarter * 32) << 16) + col;
}

// store 32 fp32 values times mul as bf16 to global row pointer + column offset
// (16-byte aligned): two 32-byte stores where the row is 32-byte aligned (a
// whole sector per lane: each lane writes a different row), else four 16-byte
__device__ __forceinline__ void store_row32(bf16* dst, const uint32_t (&r)[32], float mul = 1.0f) {
  uint4 pk[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(r[v * 8 + e]) * mul;
    pk[v] = pack8f(f);
  }
  if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + h * 16), "r"(pk[2 * h].x),
                   "r"(pk[2 * h].y), "r"(pk[2 * h].z), "r"(pk[2 * h].w), "r"(pk[2 * h + 1].x), "r"(pk[2 * h + 1].y),
                   "r"(pk[2 * h + 1].z), "r"(pk[2 * h + 1].w)
                   : "memory");
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4*>(dst + v * 8) = pk[v];
  }
}

__device__ __forceinline__ void mma_tile(uint32_t d_tmem, uint32_t a_tile, bool a_mn, uint32_t b_tile, bool b_mn,
                                         int ksteps, uint32_t idesc, bool accumulate) {
  for (int k = 0; k < ksteps; ++k) {
    const uint64_t ad = a_mn ? desc_mnmajor(a_tile, k) : desc_kmajor(a_tile, k);
    const uint64_t bd = b_mn ? desc_mnmajor(b_tile, k) : desc_kmajor(b_tile, k);
    umma_bf16(d_tmem, ad, bd, idesc, (accumulate || k > 0) ? 1u : 0u);
  }
}

__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
}

#endif

}  // namespace tp3d
