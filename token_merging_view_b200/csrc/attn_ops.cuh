// Device pieces shared by the kernels of attention over key ranges.
#pragma once
#include "attn_ops.h"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace httm {
namespace tc {

constexpr uint32_t kTileBytes = kAttnTile * kAttnD * 2;   // 16 KB: 128 rows x 64 bf16

__device__ __forceinline__ void tma_load_tile(void* dst, const AttnMap& m, uint64_t* bar, int token, int head,
                                              int batch) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(&m.map)), "r"(smem_u32(bar)), "r"(0), "r"(token), "r"(head * m.hmul),
      "r"(batch * m.bmul)
      : "memory");
}

// One lane of a converged warp, always the same one; the compiler knows the
// branch for what it is and keeps the operands of the MMAs in it uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
// A value that every lane holds, as one the compiler can treat so.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// A wait of a whole warp, with a result the compiler knows to be uniform.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, DevState* st) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, st));
}

// A plain bulk copy; addresses and size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The key range of query l of batch entry b, clamped to [0, N]; (0, 0) if empty.
__device__ __forceinline__ int2 key_range(const AttnArgs& a, int b, int l) {
  const size_t i = (size_t)b * a.L + l;
  const int lo = a.kb ? max(a.kb[i], 0) : 0, hi = a.ke ? min(a.ke[i], a.N) : a.N;
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}

// A full warp: zero the rows r < n of a swizzled tile for which dead(r) holds.
template <class F>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int n, F&& dead) {
  for (int r = threadIdx.x & 31; r < n; r += 32)
    if (dead(r)) {
#pragma unroll
      for (int c = 0; c < 8; ++c) reinterpret_cast<uint4*>(tile + r * 128)[c] = make_uint4(0, 0, 0, 0);
    }
}

// Is one of the two bf16 of x an infinity or NaN?
__device__ __forceinline__ bool wild(uint32_t x) {
  return (x & 0x7f800000u) == 0x7f800000u || (x & 0x7f80u) == 0x7f80u;
}
__device__ __forceinline__ bool wild(uint4 x) { return wild(x.x) || wild(x.y) || wild(x.z) || wild(x.w); }
__device__ __forceinline__ uint32_t tame(uint32_t x) {
  return ((x & 0x7f800000u) == 0x7f800000u ? 0u : x & 0xffff0000u) | ((x & 0x7f80u) == 0x7f80u ? 0u : x & 0xffffu);
}
// Does row r (128 bytes) of a swizzled tile hold infinities or NaN?
// Neighbouring rows start at different 16-byte chunks, so a warp's accesses
// meet no bank twice; an exponent of ones plus one carries into the sign bit.
__device__ __forceinline__ bool wild_row(const uint8_t* tile, int r) {
  const uint4* row = reinterpret_cast<const uint4*>(tile + r * 128);
  uint32_t any = 0u;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 x = row[c ^ (r & 7)];
    any |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
           ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
  }
  return (any & 0x80008000u) != 0u;
}
// They become 0.
__device__ __forceinline__ void tame_row(uint8_t* tile, int r) {
  uint4* row = reinterpret_cast<uint4*>(tile + r * 128);
  for (int c = 0; c < 8; ++c) {
    const uint4 x = row[c];
    row[c] = make_uint4(tame(x.x), tame(x.y), tame(x.z), tame(x.w));
  }
}

// Bounded wait that ignores the abort flag (to drain MMAs in flight).
__device__ __forceinline__ void drain_mma(uint64_t* bar, uint32_t parity) {
  const WaitClock clk;
  while (!mbar_try_wait(bar, parity))
    if (clk.expired()) return;
}

__device__ __forceinline__ int warp_min(int v) { return __reduce_min_sync(0xffffffffu, v); }
__device__ __forceinline__ int warp_max(int v) { return __reduce_max_sync(0xffffffffu, v); }

// 64 consecutive TMEM columns of this row (whole warp).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
  tmem_ld32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
  tmem_wait_ld();
}

// Channels [c0, c0 + 8 n) of a row below d, times f, to bf16 memory (d a
// multiple of 8).
template <int N>
__device__ __forceinline__ void store_row_bf16(const uint32_t* o, __nv_bfloat16* dst, float f, int c0, int d) {
#pragma unroll
  for (int v = 0; v < N; ++v)
    if (c0 + v * 8 < d) {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        u[e] = pack_bf16(__uint_as_float(o[v * 8 + 2 * e]) * f, __uint_as_float(o[v * 8 + 2 * e + 1]) * f);
      reinterpret_cast<uint4*>(dst + c0)[v] = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

}  // namespace tc
}  // namespace httm
