// Attention over key ranges, forward: out_i = sum_j P_ij V_j over the keys
// j in [begin_i, end_i), and the row's log-sum-exp.
//
// Query rows: the G query heads that share a key head are packed next to
// each other (row r = query r / G, head r % G), so K and V are read once for
// all of them and a single token of a grouped model fills G rows of a tile.
// A work item is up to 256 such rows of one key head -- two 128-row tiles,
// or one when there are no more -- against the union of their key ranges.
//
// Long sequences (attn_range_fwd_kernel), 12 warps: warp 0 loads K/V tiles of
// 128 keys by TMA into a ring of four; warp 1 issues tcgen05.mma (S = Q K^T
// from shared memory, then O += P V with P read from TMEM); warps 4..7 and
// 8..11 are the softmax of tiles 0 and 1, one row a thread.  TMEM: a ring of three 128-column S buffers (P
// overwrites half of its S), O_0 and O_1 of 64 columns: 512.  The i-th S
// product goes to buffer i % 3 and is issued right behind the P V product
// that frees it, so the tensor core works on one tile during the other's
// softmax.  Scores are exponentiated against a maximum in use that is raised
// (and O rescaled) only when a tile's sum passes 2^16.  Bound by the exp
// unit together with the cost of the N = 64 MMAs, as the layer's dense
// attention is.  (Up to 32 rows a key head have a kernel of their own.)
//
// Splits: with fewer items than SMs, or a last wave that would run mostly
// empty, each item's keys are cut in `parts` ranges of whole tiles; the parts
// leave unnormalised sums and maxima, which attn_join_kernel adds up in order.
//
// Roundings: scores, the running sum (of the unrounded P) and O are fp32.  P
// is rounded to bf16, at most 2^-8 of itself, because it is an operand of the
// tensor core beside a bf16 V: a second product for what the rounding takes
// off would cost half of the call again.  The result is rounded once.
//
// Masks: a tile that every row of a warp sees whole takes no compares.
// Keys outside the union of the item's ranges never enter: whole tiles are
// not loaded, and in the last tile the V rows behind the union are zeroed
// (a zero probability times a NaN there would not be zero).  In a tile that
// only some rows see, infinities and NaN in V are taken out before the
// product and added at the end to the rows that see them, so that they reach
// no other (the check costs such tiles about a tenth, other tiles nothing).
#include <algorithm>

#include "attn_ops.cuh"

namespace httm {
namespace {

using namespace tc;

constexpr int kStages = 4;
constexpr int kThreads = 384;
constexpr int kAuxRegs = 88, kSoftmaxRegs = 208;   // of 384 x 168 at launch
constexpr uint32_t kColO = 384;           // O_t at kColO + 64 t; S ring at 0, 128, 256
constexpr int kPartStride = httm::kAttnRangePart;

// Where V held infinities or NaN in a tile with masks: mark i is set for some
// of the part's keys i, i + kWildMarks, ...
constexpr int kWildMarks = 4096;          // 16 a thread of the smaller block
struct WildKeys {
  alignas(16) uint8_t mark[kWildMarks];
  int any;
};

struct FwdSmem {
  uint8_t q[2][kTileBytes];
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  uint64_t q_full;
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[3], p_full[2], o_done[2];
  uint64_t drain, dirty, clean;
  int lo[8], hi[8], f_lo[8], f_hi[8];
  uint32_t tmem_base;
  int abort;
  WildKeys wild;
};
constexpr size_t kSmemBytes = sizeof(FwdSmem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Adds the infinities and NaN of the marked values, `n` keys of the part from
// `base` on, to the output row of a thread that sees `keys`.  A warp's lanes
// walk together, so that their loads are broadcasts; out of line, where it
// costs the kernel no registers.
template <class T>
__device__ __noinline__ void add_wild(const AttnArgs& a, int b, int kh, const WildKeys& w, int base, int n, int2 keys,
                                      T* row) {
  const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.v.data) + b * a.v.sb + kh * a.v.sh;
  const int end = min(base + n, a.N);
  for (int c = 0; c < a.d; c += 8) {
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < min(n, kWildMarks); i += 16) {
      const uint4 marks = *reinterpret_cast<const uint4*>(w.mark + i);
      if ((marks.x | marks.y | marks.z | marks.w) == 0u) continue;
      for (int at = i; at < i + 16; ++at)
        for (int key = w.mark[at] ? base + at : end; key < end; key += kWildMarks) {
          const uint4 x = *reinterpret_cast<const uint4*>(v + (int64_t)key * a.v.st + c);
          if (!wild(x) || key < keys.x || key >= keys.y) continue;
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float f = __uint_as_float((e & 1) ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
            if (!isfinite(f)) sum[e] += f;
          }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!isfinite(sum[e])) row[c + e] = from_f<T>(to_f(row[c + e]) + sum[e]);
  }
}

// A query row into the swizzled tile (zeros behind d, and for rows that see
// nothing, whatever memory holds there).
__device__ __forceinline__ void load_query_row(const AttnArgs& a, uint8_t* tile, int row, int b, int head, int l, bool live) {
  const __nv_bfloat16* src =
      reinterpret_cast<const __nv_bfloat16*>(a.q.data) + b * a.q.sb + head * a.q.sh + (int64_t)l * a.q.st;
  uint8_t* dst = tile + row * 128;
  uint4 x[8];
#pragma unroll
  for (int c = 0; c < 8; ++c)
    x[c] = live && c * 8 < a.d ? reinterpret_cast<const uint4*>(src)[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int c = 0; c < 8; ++c) reinterpret_cast<uint4*>(dst)[c ^ (row & 7)] = x[c];
}

// A finished row: to `part` its unnormalised sums, the row sum and the
// maximum in use, or (part null) the output and its log-sum-exp.  `o` is its O
// if it has any; `w`: see add_wild.
__device__ __forceinline__ void finish_row(const AttnArgs& a, int b, int kh, int head, int l, bool in_item, bool live,
                                           bool any, const uint32_t (&o)[64], float sum, float m_used, float* part,
                                           const WildKeys& w, int base, int n, int2 keys) {
  if (!in_item) return;
  if (part) {
    if (any) {
#pragma unroll
      for (int v = 0; v < 16; ++v)
        reinterpret_cast<float4*>(part)[v] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                         __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
    }
    part[kAttnD] = sum;
    part[kAttnD + 1] = m_used;
    if (w.any) add_wild(a, b, kh, w, base, n, keys, part);
    return;
  }
  __nv_bfloat16* dst =
      reinterpret_cast<__nv_bfloat16*>(a.out.data) + b * a.out.sb + head * a.out.sh + (int64_t)l * a.out.st;
  // a row that saw nothing has P = 0 in every step or was never written: its
  // output is 0 by definition
  if (any && live) {
    store_row_bf16<8>(o, dst, 1.f / sum, 0, a.d);
  } else {
    for (int v = 0; v < a.d / 8; ++v) reinterpret_cast<uint4*>(dst)[v] = make_uint4(0, 0, 0, 0);
  }
  if (w.any) add_wild(a, b, kh, w, base, n, keys, dst);
  if (a.lse)
    a.lse[((size_t)b * a.H + head) * a.L + l] = live ? (m_used + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
}

__global__ void __launch_bounds__(kThreads, 1)
attn_range_fwd_kernel(const __grid_constant__ AttnMap mk, const __grid_constant__ AttnMap mv,
                      const __grid_constant__ AttnArgs a, int row_tiles, int parts, float* __restrict__ part_out) {
  extern __shared__ uint8_t smem_raw[];
  FwdSmem& sm = *reinterpret_cast<FwdSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  // later rows usually see more keys (causal): they go first
  const unsigned item = blockIdx.x / parts, part = blockIdx.x % parts;
  const int bk = item / row_tiles, rt = row_tiles - 1 - item % row_tiles;
  const int b = bk / a.K, kh = bk % a.K;
  const int rows = a.L * a.G - rt * 256;             // rows from this item's first on
  const int n_t = rows > 128 ? 2 : 1;
  DevState* st = a.st;

  // this thread's query row (softmax threads): its head, query and keys
  const int t = warp >= 8 ? 1 : 0;
  const int row = (warp & 3) * 32 + lane;            // row inside the tile = TMEM lane
  const int r_item = t * 128 + row;
  const bool in_item = warp >= 4 && r_item < rows;
  const int r_all = rt * 256 + r_item;
  const int l = in_item ? r_all / a.G : 0, head = in_item ? kh * a.G + (r_all - l * a.G) : 0;
  int2 keys = in_item ? key_range(a, b, l) : make_int2(0, 0);
  if (warp >= 4) {
    const bool live = keys.x < keys.y;
    const int lo = warp_min(live ? keys.x : 0x7fffffff), hi = warp_max(live ? keys.y : 0);
    const int f_lo = warp_max(live ? keys.x : 0), f_hi = warp_min(live ? keys.y : 0x7fffffff);
    if (lane == 0) {
      sm.lo[warp - 4] = lo;
      sm.hi[warp - 4] = hi;
      sm.f_lo[warp - 4] = f_lo;
      sm.f_hi[warp - 4] = f_hi;
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 128 * n_t);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&sm.s_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.o_done[i], 1);
    }
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.dirty, 1);
    mbar_init(&sm.clean, 1);
    sm.abort = 0;
    sm.wild.any = 0;
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(&sm.tmem_base, 512);
  if (threadIdx.x < kWildMarks / 16) reinterpret_cast<uint4*>(sm.wild.mark)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  int lo = 0x7fffffff, hi = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = min(lo, sm.lo[i]);
    hi = max(hi, sm.hi[i]);
  }
  // this part's tiles: keys [base, base + 128 n_kv) of [lo, hi)
  const int n_all = hi > lo ? (hi - lo + kAttnTile - 1) / kAttnTile : 0;
  const int j0 = (int)((long long)n_all * part / parts);
  const int n_kv = uniform((int)((long long)n_all * (part + 1) / parts) - j0);
  const int base = n_all > 0 ? lo + j0 * kAttnTile : 0;
  const int n_last = hi - (base + (n_kv - 1) * kAttnTile);   // keys of the union in the last tile

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAuxRegs) : "memory");
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ producer
      for (int j = 0; j < n_kv; ++j) {
        const int s = j % kStages;
        if (j >= kStages && !mbar_wait(&sm.kv_empty[s], ((j / kStages) - 1) & 1, abort, st)) break;
        mbar_arrive_expect_tx(&sm.kv_full[s], 2 * kTileBytes);
        tma_load_tile(sm.k[s], mk, &sm.kv_full[s], base + j * kAttnTile, kh, b);
        tma_load_tile(sm.v[s], mv, &sm.kv_full[s], base + j * kAttnTile, kh, b);
      }
    } else if (warp == 1 && n_kv > 0) {
      // ------------------------------------------------------------ MMA issue
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t id_o = idesc_bf16(128, kAttnD, false, true);
      const int n_prod = n_t * n_kv;                 // S products: i = n_t j + tile
      const uint64_t qd = sw128_desc(smem_u32(sm.q[0]), 1024), kd = sw128_desc(smem_u32(sm.k[0]), 1024),
                     vd = sw128_desc(smem_u32(sm.v[0]), 1024);
      constexpr uint64_t kNext = kTileBytes >> 4;    // from one tile's descriptor to the next one's
      // product i: waits for its K/V tile if it is the tile's first
      auto issue_qk = [&](int i) -> bool {
        const int j = n_t == 2 ? i >> 1 : i, tile = n_t == 2 ? i & 1 : 0, s = j % kStages;
        if (tile == 0) {
          if (!wait_all(&sm.kv_full[s], (j / kStages) & 1, abort, st)) return false;
          if (j == n_kv - 1 && n_last < kAttnTile) {
            if (lane == 0) mbar_arrive(&sm.dirty);
            if (!wait_all(&sm.clean, 0, abort, st)) return false;
          }
          tc_fence_after();
        }
        const uint64_t A = qd + tile * kNext, B = kd + s * kNext;
        const uint32_t col = tmem + (i % 3) * 128;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kAttnD / 16; ++kk) umma_bf16(col, A + kk * 2, B + kk * 2, id_s, kk > 0);
          umma_commit(&sm.s_full[i % 3]);
        }
        __syncwarp();
        return true;
      };
      bool ok = wait_all(&sm.q_full, 0, abort, st);
      for (int i = 0; ok && i < min(3, n_prod); ++i) ok = issue_qk(i);
      for (int i = 0; ok && i < n_prod; ++i) {
        const int j = n_t == 2 ? i >> 1 : i, tile = n_t == 2 ? i & 1 : 0, s = j % kStages;
        if (!wait_all(&sm.p_full[tile], j & 1, abort, st)) break;
        tc_fence_after();
        const uint64_t B = vd + s * kNext;
        const uint32_t pc = tmem + (i % 3) * 128, oc = tmem + kColO + tile * 64;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kAttnTile / 16; ++kk)
            umma_bf16_ts(oc, pc + kk * 8, B + kk * 128, id_o, (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&sm.o_done[tile]);
          if (tile == n_t - 1) umma_commit(&sm.kv_empty[s]);
        }
        __syncwarp();
        if (i + 3 < n_prod) ok = issue_qk(i + 3);
      }
      if (elect_one()) {
        umma_commit(&sm.drain);                      // every MMA ends before TMEM is released
        drain_mma(&sm.drain, 0);
      }
      __syncwarp();
    } else if (warp == 2 && n_kv > 0 && n_last < kAttnTile) {
      // ------------------------------------------------------------ V rows behind the union of the ranges
      const int s = (n_kv - 1) % kStages;
      if (__all_sync(0xffffffffu, mbar_wait(&sm.dirty, 0, abort, st)) &&
          __all_sync(0xffffffffu, mbar_wait(&sm.kv_full[s], ((n_kv - 1) / kStages) & 1, abort, st))) {
        zero_rows(sm.v[s], kAttnTile, [&](int r) { return r >= n_last; });
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.clean);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs) : "memory");
    // -------------------------------------------------------------- softmax
    if (t < n_t) {
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t to = tmem + lane_off + kColO + t * 64;      // this row of O_t
      const bool live = keys.x < keys.y;
      const bool warp_live = __any_sync(0xffffffffu, live);
      // the warp's keys: some row sees [w_lo, w_hi), every live row [f_lo,
      // f_hi); every live row of the tile [t_lo, t_hi)
      // (warp reductions: the compiler knows their results to be uniform)
      const int w_lo = warp_min(live ? keys.x : 0x7fffffff) - base, w_hi = warp_max(live ? keys.y : 0) - base;
      const int f_lo = warp_max(live ? keys.x : 0) - base, f_hi = warp_min(live ? keys.y : 0x7fffffff) - base;
      const int t_lo = warp_max(sm.f_lo[t * 4 + (lane & 3)]) - base;
      const int t_hi = max(warp_min(sm.f_hi[t * 4 + (lane & 3)]), 0) - base;
      load_query_row(a, sm.q[t], row, b, head, l, live);
      fence_async_smem();
      mbar_arrive(&sm.q_full);
      float m_used = -INFINITY, sum = 0.f;
      bool ok = true;
      for (int j = 0; j < n_kv; ++j) {
        const int i = n_t * j + t, buf = i % 3;                  // S product and its ring buffer
        const uint32_t ts = tmem + lane_off + buf * 128;         // this row of S, then of P
        // waits are made warp-uniform: tcgen05.ld/st below need every lane
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[buf], (i / 3) & 1, abort, st))) { ok = false; break; }
        tc_fence_after();
        const int k0 = j * kAttnTile;                            // the tile's keys, counted from base
        bool pv_done = j == 0;                                   // PV(t, j-1) seen complete
        if (t_lo > k0 || t_hi < min(k0 + kAttnTile, hi - base)) {
          // some row does not see all that others see of this tile, and its
          // zero probability times an infinity or NaN there would not be
          // zero: those elements leave V (one row a thread) and reach the
          // rows that do see them at the end
          const int s = j % kStages;
          if (!__all_sync(0xffffffffu, mbar_wait(&sm.kv_full[s], (j / kStages) & 1, abort, st))) { ok = false; break; }
          if (wild_row(sm.v[s], row)) {
            // tile 0's product with this V comes first and takes it as it
            // is; tile 1's comes behind both tiles' P, so it sees the note
            if (t == 1) mbar_wait(&sm.o_done[0], j & 1, abort, st);
            sm.wild.mark[(k0 + row) % kWildMarks] = 1;
            sm.wild.any = 1;
            tame_row(sm.v[s], row);
            fence_async_smem();
          }
        }
        if (w_lo >= k0 + kAttnTile || w_hi <= k0) {
          // none of this warp's rows sees this tile: P = 0 (rows that are
          // never stored may keep what is there)
          if (warp_live) {
            uint32_t z[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) z[e] = 0u;
            tmem_st32(ts, z);
            tmem_st32(ts + 32, z);
          }
        } else {
          uint32_t sr[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
          tmem_wait_ld();
          if (f_lo > k0 || f_hi < k0 + kAttnTile) {
            const int first = keys.x - base - k0, last = keys.y - base - k0;
#pragma unroll
            for (int e = 0; e < kAttnTile; ++e)
              if (e < first || e >= last) sr[e] = __float_as_uint(-INFINITY);
          }
          // p = 2^(s c - m) against the maximum in use.  Sums above 2^16
          // (always so on a row's first tile, where m = -inf) make the warp
          // raise the maximum, rescale O and the sum, and redo the tile.
          const unsigned long long cc = f2_pack(a.scale_log2, a.scale_log2);
          float rsum = 0.f, m_ref = m_used;
          for (int pass = 0; pass < 2; ++pass) {
            const unsigned long long mm = f2_pack(-m_ref, -m_ref);
            unsigned long long rs[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) rs[e] = 0ull;            // (0.f, 0.f)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t pk[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float s0 = __uint_as_float(sr[c * 64 + 2 * e]), s1 = __uint_as_float(sr[c * 64 + 2 * e + 1]);
                const unsigned long long xp = f2_fma(f2_pack(s0, s1), cc, mm);
                float x0, x1;
                f2_unpack(xp, x0, x1);
                const float p0 = ex2(x0), p1 = ex2(x1);
                rs[e & 3] = f2_add(rs[e & 3], f2_pack(p0, p1));
                pk[e] = pack_bf16(p0, p1);
              }
              tmem_st32(ts + c * 32, pk);
            }
            float r0, r1, r2, r3, r4, r5, r6, r7;
            f2_unpack(rs[0], r0, r1);
            f2_unpack(rs[1], r2, r3);
            f2_unpack(rs[2], r4, r5);
            f2_unpack(rs[3], r6, r7);
            rsum = ((r0 + r1) + (r2 + r3)) + ((r4 + r5) + (r6 + r7));
            if (pass == 1) break;
            // rows that see nothing never ask; NaN sums count as large
            const bool need = live && !(rsum <= 65536.f);
            if (!__any_sync(0xffffffffu, need)) break;
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 64; ++e)
              mx[e & 3] = max3(mx[e & 3], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
            // a row that did not ask keeps its reference, and so its bits
            const float m_new = need ? fmaxf(m_used, max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * a.scale_log2) : m_used;
            // a row with nothing yet: reference 0, its P and sum stay 0
            m_ref = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = m_used == -INFINITY ? 0.f : ex2(m_used - m_ref);
            if (j > 0) {
              if (!__all_sync(0xffffffffu, mbar_wait(&sm.o_done[t], (j - 1) & 1, abort, st))) {
                ok = false;
                break;
              }
              pv_done = true;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t o[32];
                tmem_ld32(to + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(to + c * 32, o);
              }
            }
            sum *= alpha;
            m_used = m_new;
          }
          if (!ok) break;
          sum += rsum;
        }
        // no arrival for step j before PV(t, j-1) is complete: every parity
        // wait on o_done is then at most one phase behind, and no warp can
        // arrive twice before a slower one of its warpgroup arrives once
        if (!pv_done && !__all_sync(0xffffffffu, mbar_wait(&sm.o_done[t], (j - 1) & 1, abort, st))) {
          ok = false;
          break;
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sm.p_full[t]);
      }
      if (ok && n_kv > 0)
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_done[t], (n_kv - 1) & 1, abort, st));
      tc_fence_after();
      if (ok) {
        uint32_t o[64];
        if (n_kv > 0) tmem_ld64(to, o);
        float* part_row =
            parts > 1 ? part_out + ((size_t)blockIdx.x * min(a.L * a.G, 256) + (in_item ? r_item : 0)) * kPartStride
                      : nullptr;
        finish_row(a, b, kh, head, l, in_item, live, n_kv > 0, o, sum, m_used, part_row, sm.wild, base, n_kv * kAttnTile,
                   keys);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (*abort) {
      // let TMA copies still in flight land before the shared memory goes away
      for (int i = 0; i < 200; ++i) __nanosleep(1000);
    }
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ two blocks an SM
// The same for shorter sequences: an item is one tile of 128 rows, and two
// blocks share an SM, each with half of the tensor memory -- two S buffers of
// 96 keys and O, 64 columns -- and of the shared memory.  The blocks hide each
// other's start and end (about 5 us a block of the kernel above) and the
// items are finer.  Two warpgroups: the helpers (K/V loads, MMA issue, V
// rows) and the softmax, one row a thread.  S products run two steps ahead;
// P and "P V done" have two barriers each, for even and odd steps: step j + 2
// is reached only behind S of j + 2, which is issued behind P V of j, so no
// barrier gets an arrival early or is two phases from a wait on it.
constexpr int kPairKeys = 96, kPairStages = 3, kPairThreads = 256;
constexpr int kPairAux = 48, kPairSoft = 208;        // registers, of 256 x 128 at launch
constexpr uint32_t kPairBytes = kPairKeys * kAttnD * 2, kPairO = 2 * kPairKeys;

struct PairSmem {
  uint8_t q[kTileBytes];
  uint8_t k[kPairStages][kPairBytes], v[kPairStages][kPairBytes];
  uint64_t q_full, kv_full[kPairStages], kv_empty[kPairStages];
  uint64_t s_full[2], p_full[2], o_done[2], drain, dirty, clean;
  int lo[4], hi[4], f_lo[4], f_hi[4];
  uint32_t tmem_base;
  int abort;
  WildKeys wild;
};
constexpr size_t kPairSmem = sizeof(PairSmem) + 1024;
static_assert(2 * (kPairSmem + 1024) <= 227 * 1024, "two blocks an SM");

__global__ void __launch_bounds__(kPairThreads, 2)
attn_range_pair_kernel(const __grid_constant__ AttnMap mk, const __grid_constant__ AttnMap mv,
                       const __grid_constant__ AttnArgs a, int row_tiles, int parts, float* __restrict__ part_out) {
  extern __shared__ uint8_t smem_raw[];
  PairSmem& sm = *reinterpret_cast<PairSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  // later rows usually see more keys (causal): they go first
  const unsigned item = blockIdx.x / parts, part = blockIdx.x % parts;
  const int bk = item / row_tiles, rt = row_tiles - 1 - item % row_tiles;
  const int b = bk / a.K, kh = bk % a.K;
  DevState* st = a.st;

  // this thread's query row (softmax threads): its head, query and keys
  const int row = (warp & 3) * 32 + lane;            // row inside the tile = TMEM lane
  const int r_all = rt * kAttnTile + row;
  const bool in_item = warp >= 4 && r_all < a.L * a.G;
  const int l = in_item ? r_all / a.G : 0, head = in_item ? kh * a.G + (r_all - l * a.G) : 0;
  const int2 keys = in_item ? key_range(a, b, l) : make_int2(0, 0);
  const bool live = keys.x < keys.y;
  if (warp >= 4) {
    const int lo = warp_min(live ? keys.x : 0x7fffffff), hi = warp_max(live ? keys.y : 0);
    const int f_lo = warp_max(live ? keys.x : 0), f_hi = warp_min(live ? keys.y : 0x7fffffff);
    if (lane == 0) {
      sm.lo[warp - 4] = lo;
      sm.hi[warp - 4] = hi;
      sm.f_lo[warp - 4] = f_lo;
      sm.f_hi[warp - 4] = f_hi;
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 128);
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.o_done[i], 1);
    }
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.dirty, 1);
    mbar_init(&sm.clean, 1);
    sm.abort = 0;
    sm.wild.any = 0;
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(&sm.tmem_base, 256);
  if (threadIdx.x < kWildMarks / 16) reinterpret_cast<uint4*>(sm.wild.mark)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  const int lo = warp_min(sm.lo[lane & 3]), hi = warp_max(sm.hi[lane & 3]);
  // this part's steps: keys [base, base + 96 n) of [lo, hi)
  const int n_all = hi > lo ? (hi - lo + kPairKeys - 1) / kPairKeys : 0;
  const int j0 = (int)((long long)n_all * part / parts);
  const int n = uniform((int)((long long)n_all * (part + 1) / parts) - j0);
  const int base = n_all > 0 ? lo + j0 * kPairKeys : 0;
  const int n_last = hi - (base + (n - 1) * kPairKeys);   // keys of the union in the last step

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairAux) : "memory");
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ producer
      for (int j = 0; j < n; ++j) {
        const int s = j % kPairStages;
        if (j >= kPairStages && !mbar_wait(&sm.kv_empty[s], ((j / kPairStages) - 1) & 1, abort, st)) break;
        mbar_arrive_expect_tx(&sm.kv_full[s], 2 * kPairBytes);
        tma_load_tile(sm.k[s], mk, &sm.kv_full[s], base + j * kPairKeys, kh, b);
        tma_load_tile(sm.v[s], mv, &sm.kv_full[s], base + j * kPairKeys, kh, b);
      }
    } else if (warp == 1 && n > 0) {
      // ------------------------------------------------------------ MMA issue
      constexpr uint32_t id_s = idesc_bf16(128, kPairKeys, false, false);
      constexpr uint32_t id_o = idesc_bf16(128, kAttnD, false, true);
      const uint64_t qd = sw128_desc(smem_u32(sm.q), 1024), kd = sw128_desc(smem_u32(sm.k[0]), 1024),
                     vd = sw128_desc(smem_u32(sm.v[0]), 1024);
      constexpr uint64_t kNext = kPairBytes >> 4;    // from one stage's descriptor to the next one's
      auto issue_qk = [&](int j) -> bool {
        const int s = j % kPairStages;
        if (!wait_all(&sm.kv_full[s], (j / kPairStages) & 1, abort, st)) return false;
        if (j == n - 1 && n_last < kPairKeys) {
          if (lane == 0) mbar_arrive(&sm.dirty);
          if (!wait_all(&sm.clean, 0, abort, st)) return false;
        }
        tc_fence_after();
        const uint64_t B = kd + s * kNext;
        const uint32_t col = tmem + (j & 1) * kPairKeys;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kAttnD / 16; ++kk) umma_bf16(col, qd + kk * 2, B + kk * 2, id_s, kk > 0);
          umma_commit(&sm.s_full[j & 1]);
        }
        __syncwarp();
        return true;
      };
      bool ok = wait_all(&sm.q_full, 0, abort, st);
      for (int j = 0; ok && j < min(2, n); ++j) ok = issue_qk(j);
      for (int j = 0; ok && j < n; ++j) {
        const int s = j % kPairStages;
        const uint64_t B = vd + s * kNext;
        const uint32_t pc = tmem + (j & 1) * kPairKeys, oc = tmem + kPairO;
        if (!wait_all(&sm.p_full[j & 1], (j >> 1) & 1, abort, st)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kPairKeys / 16; ++kk)
            umma_bf16_ts(oc, pc + kk * 8, B + kk * 128, id_o, (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&sm.o_done[j & 1]);
          umma_commit(&sm.kv_empty[s]);
        }
        __syncwarp();
        if (j + 2 < n) ok = issue_qk(j + 2);
      }
      if (elect_one()) {
        umma_commit(&sm.drain);                      // every MMA ends before TMEM is released
        drain_mma(&sm.drain, 0);
      }
      __syncwarp();
    } else if (warp == 2 && n > 0 && n_last < kPairKeys) {
      // ------------------------------------------------------------ V rows behind the union of the ranges
      const int s = (n - 1) % kPairStages;
      if (wait_all(&sm.dirty, 0, abort, st) && wait_all(&sm.kv_full[s], ((n - 1) / kPairStages) & 1, abort, st)) {
        zero_rows(sm.v[s], kPairKeys, [&](int r) { return r >= n_last; });
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.clean);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairSoft) : "memory");
    // -------------------------------------------------------------- softmax
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lane_off + kPairO;                // this row of O
    const bool warp_live = __any_sync(0xffffffffu, live);
    const int w_lo = warp_min(live ? keys.x : 0x7fffffff) - base, w_hi = warp_max(live ? keys.y : 0) - base;
    const int f_lo = warp_max(live ? keys.x : 0) - base, f_hi = warp_min(live ? keys.y : 0x7fffffff) - base;
    const int t_lo = warp_max(sm.f_lo[lane & 3]) - base, t_hi = warp_min(sm.f_hi[lane & 3]) - base;
    load_query_row(a, sm.q, row, b, head, l, live);
    fence_async_smem();
    mbar_arrive(&sm.q_full);
    float m_used = -INFINITY, sum = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const uint32_t ts = tmem + lane_off + (j & 1) * kPairKeys; // this row of S, then of P
      // waits are made warp-uniform: tcgen05.ld/st below need every lane
      if (!wait_all(&sm.s_full[j & 1], (j >> 1) & 1, abort, st)) { ok = false; break; }
      tc_fence_after();
      const int k0 = j * kPairKeys;                              // the step's keys, counted from base
      if (t_lo > k0 || t_hi < min(k0 + kPairKeys, hi - base)) {
        // a row does not see all that others see: no infinities or NaN in V
        const int s = j % kPairStages;
        if (!wait_all(&sm.kv_full[s], (j / kPairStages) & 1, abort, st)) { ok = false; break; }
        if (row < kPairKeys && wild_row(sm.v[s], row)) {
          sm.wild.mark[(k0 + row) % kWildMarks] = 1;
          sm.wild.any = 1;
          tame_row(sm.v[s], row);
          fence_async_smem();
        }
      }
      if (w_lo >= k0 + kPairKeys || w_hi <= k0) {
        // none of this warp's rows sees this step: P = 0 (rows that are never
        // stored may keep what is there)
        if (warp_live) {
          uint32_t z[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll
          for (int c = 0; c < kPairKeys / 2; c += 16) tmem_st16(ts + c, z);
        }
      } else {
        uint32_t sr[kPairKeys];
#pragma unroll
        for (int c = 0; c < kPairKeys; c += 32) tmem_ld32(ts + c, *reinterpret_cast<uint32_t(*)[32]>(&sr[c]));
        tmem_wait_ld();
        if (f_lo > k0 || f_hi < k0 + kPairKeys) {
          const int first = keys.x - base - k0, last = keys.y - base - k0;
#pragma unroll
          for (int e = 0; e < kPairKeys; ++e)
            if (e < first || e >= last) sr[e] = __float_as_uint(-INFINITY);
        }
        // p = 2^(s c - m) against the maximum in use, as above
        const unsigned long long cc = f2_pack(a.scale_log2, a.scale_log2);
        float rsum = 0.f, m_ref = m_used;
        for (int pass = 0; pass < 2; ++pass) {
          const unsigned long long mm = f2_pack(-m_ref, -m_ref);
          unsigned long long rs[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) rs[e] = 0ull;              // (0.f, 0.f)
#pragma unroll
          for (int c = 0; c < kPairKeys; c += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c + 2 * e]), __uint_as_float(sr[c + 2 * e + 1])), cc, mm), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              rs[e & 3] = f2_add(rs[e & 3], f2_pack(p0, p1));
              pk[e] = pack_bf16(p0, p1);
            }
            tmem_st16(ts + c / 2, pk);
          }
          float r0, r1, r2, r3, r4, r5, r6, r7;
          f2_unpack(rs[0], r0, r1);
          f2_unpack(rs[1], r2, r3);
          f2_unpack(rs[2], r4, r5);
          f2_unpack(rs[3], r6, r7);
          rsum = ((r0 + r1) + (r2 + r3)) + ((r4 + r5) + (r6 + r7));
          if (pass == 1) break;
          const bool need = live && !(rsum <= 65536.f);
          if (!__any_sync(0xffffffffu, need)) break;
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kPairKeys / 2; ++e)
            mx[e & 3] = max3(mx[e & 3], __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
          // a row that did not ask keeps its reference, and so its bits
          const float m_new = need ? fmaxf(m_used, max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * a.scale_log2) : m_used;
          m_ref = m_new == -INFINITY ? 0.f : m_new;
          const float alpha = m_used == -INFINITY ? 0.f : ex2(m_used - m_ref);
          if (j > 0) {
            if (!wait_all(&sm.o_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort, st)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t o[32];
              tmem_ld32(to + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(to + c * 32, o);
            }
          }
          sum *= alpha;
          m_used = m_new;
        }
        if (!ok) break;
        sum += rsum;
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.p_full[j & 1]);
    }
    if (ok && n > 0) ok = wait_all(&sm.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort, st);
    tc_fence_after();
    if (ok) {
      uint32_t o[64];
      if (n > 0) tmem_ld64(to, o);
      float* part_row = parts > 1 ? part_out + ((size_t)blockIdx.x * min(a.L * a.G, kAttnTile) + (in_item ? row : 0)) * kPartStride
                                  : nullptr;
      finish_row(a, b, kh, head, l, in_item, live, n > 0, o, sum, m_used, part_row, sm.wild, base, n * kPairKeys, keys);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (*abort)
      for (int i = 0; i < 200; ++i) __nanosleep(1000);           // copies in flight land
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// Adds up the parts of every row: with M the largest maximum in use, O =
// sum_p O_p 2^(m_p - M) / sum_p l_p 2^(m_p - M), in part order.  16 threads
// a row, four channels each.
__global__ void __launch_bounds__(256)
attn_join_kernel(const __grid_constant__ AttnArgs a, int tile_rows, int row_tiles, int parts,
                 const float* __restrict__ part_in) {
  const int rows = a.L * a.G, item_rows = min(rows, tile_rows);
  const long long idx = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (idx >= (long long)a.B * a.K * rows) return;
  const int c = threadIdx.x & 15;
  const int bk = (int)(idx / rows), r = (int)(idx % rows), rt = r / tile_rows;
  const long long item = (long long)bk * row_tiles + (row_tiles - 1 - rt);
  const float* src = part_in + ((size_t)item * parts * item_rows + (r - rt * tile_rows)) * kPartStride;
  const size_t step = (size_t)item_rows * kPartStride;
  float mx = -INFINITY, sum = 0.f;
  for (int p = 0; p < parts; ++p) mx = fmaxf(mx, src[p * step + kAttnD + 1]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < parts; ++p) {
    const float m = src[p * step + kAttnD + 1], l = src[p * step + kAttnD];
    // saw none of its keys, and may have left no O.  (Maxima pass NaN over: a
    // part whose scores are all NaN has this maximum too, and a sum of NaN.)
    if (m == -INFINITY && l == 0.f) continue;
    const float w = ex2(m - mx);
    const float4 x = reinterpret_cast<const float4*>(src + p * step)[c];
    sum = fmaf(l, w, sum);
    o.x = fmaf(x.x, w, o.x), o.y = fmaf(x.y, w, o.y), o.z = fmaf(x.z, w, o.z), o.w = fmaf(x.w, w, o.w);
  }
  const int l = r / a.G, head = (bk % a.K) * a.G + (r - l * a.G), b = bk / a.K;
  const int2 keys = key_range(a, b, l);
  const bool live = keys.x < keys.y;
  const float inv = live ? 1.f / sum : 0.f;
  if (!live) o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c * 4 < a.d) {
    __nv_bfloat16* dst =
        reinterpret_cast<__nv_bfloat16*>(a.out.data) + b * a.out.sb + head * a.out.sh + (int64_t)l * a.out.st;
    reinterpret_cast<uint2*>(dst)[c] = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  }
  if (c == 0 && a.lse)
    a.lse[((size_t)b * a.H + head) * a.L + l] = live ? (mx + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

namespace {
// One kernel's plan: in how many parts each item's keys are cut, by a count of
// time in the large kernel's steps (256 rows, 128 keys: 1.5 us).  A step of 96
// keys takes 0.77 in a block of the pair kernel, 0.55 if the block has its SM
// for itself; a block's start and end take 4 in either, a join 4 for its
// launch and its share of the partial rows.
void split(const httm_attention& a, bool pair, AttnFwdPlan* p) {
  const int keys = pair ? kPairKeys : kAttnTile, slots = pair ? 2 * kSMs : kSMs;
  p->pair = pair;
  p->tile_rows = pair ? kAttnTile : 2 * kAttnTile;
  p->row_tiles = (p->rows + p->tile_rows - 1) / p->tile_rows;
  const long long heads = (long long)a.batch * a.kv_heads, steps = ((long long)a.kv_len + keys - 1) / keys;
  p->items = heads * p->row_tiles;
  p->parts = 1;
  double best = 0;
  for (long long n = 1; n <= std::min<long long>(kAttnMaxParts, std::max(1ll, steps)); ++n) {
    if (n > 1 && p->items * n > 16 * slots) break;
    const long long full = p->items * n / slots, rest = p->items * n % slots, each = (steps + n - 1) / n;
    const double step = pair ? 0.77 : 1.0, last = pair && rest <= kSMs ? 0.55 : step;
    const double join = n > 1 ? 4 + (double)p->rows * heads * n * 1.2e-4 : 0;
    const double cost = full * (each * step + 4) + (rest ? each * last + 4 : 0) + join;
    if (n == 1 || cost < best) {
      best = cost;
      p->parts = (int)n;
    }
  }
}
}  // namespace

// Which kernel: the pair kernel up to 8,192 keys.  Measured with 16 heads,
// large kernel against pair: 64 x 128 tokens 52 and 35 us, 32 x 256 47 and 41,
// 8 x 1,369 149 and 127, 2 x 2,738 131 and 111, 8,214 423 and 421, 16,384 1345
// and 1390.  Split (one sequence): 64 queries on 1,369 keys 14.8 and 13.1, on
// 8,000 20.9 and 22.5; 317 on 2,738 25.0 and 20.5, on 8,000 39.7 and 31.8; with
// 4 key heads 64 on 1,369 20.0 and 13.9, on 8,000 27.2 and 20.5.  Over 34 to
// 1,000 queries on 500 to 8,000 keys the large one is 12 % behind in the mean,
// 44 % at most, and at most 15 % ahead (64 on 5,476, 18.5 and 21.3).
AttnFwdPlan attn_fwd_plan(const httm_attention& a, bool ranges) {
  AttnFwdPlan p{};
  p.rows = a.q_len * (a.heads / a.kv_heads);
  p.few = p.rows <= kAttnFewRows;
  if (p.few) {
    p.tile_rows = 2 * kAttnTile;
    p.row_tiles = 1;
    p.items = (long long)a.batch * a.kv_heads;
    p.parts = attn_rows_parts(a, ranges);
  } else {
    split(a, a.kv_len <= 8192, &p);
  }
  p.part_bytes = p.parts > (p.few ? kAttnCluster : 1)
                     ? (size_t)p.items * p.parts * std::min(p.rows, p.tile_rows) * kPartStride * 4 : 0;
  return p;
}

namespace {
cudaError_t launch_join(const AttnArgs& a, const AttnFwdPlan& p, const float* part, cudaStream_t s) {
  if (p.parts == 1) return cudaSuccess;
  const long long rows = (long long)a.B * a.K * p.rows;
  attn_join_kernel<<<(unsigned)((rows + 15) / 16), 256, 0, s>>>(a, p.tile_rows, p.row_tiles, p.parts, part);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_attn_fwd(const AttnArgs& a, const AttnFwdPlan& p, void* ws, cudaStream_t s) {
  float* part = static_cast<float*>(ws);
  if (p.few) {
    const cudaError_t e = launch_attn_rows(a, p, part, s);
    return e != cudaSuccess || p.parts <= kAttnCluster ? e : launch_join(a, p, part, s);
  }
  AttnMap mk, mv;
  const int keys = p.pair ? kPairKeys : kAttnTile;
  // without keys nothing is loaded through their maps
  if (!attn_map(&mk, a.k, a.q.data, a.d, a.N, a.K, a.B, keys) || !attn_map(&mv, a.v, a.q.data, a.d, a.N, a.K, a.B, keys))
    return cudaErrorInvalidValue;
  if (p.pair) {
    cudaError_t e = check_registers<attn_range_pair_kernel>(kPairThreads, 128 * kPairAux + 128 * kPairSoft);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attn_range_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem);
    if (e != cudaSuccess) return e;
    attn_range_pair_kernel<<<(unsigned)(p.items * p.parts), kPairThreads, kPairSmem, s>>>(mk, mv, a, p.row_tiles,
                                                                                         p.parts, part);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join(a, p, part, s);
  }
  cudaError_t e = check_registers<attn_range_fwd_kernel>(kThreads, 128 * kAuxRegs + 256 * kSoftmaxRegs);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attn_range_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  attn_range_fwd_kernel<<<(unsigned)(p.items * p.parts), kThreads, kSmemBytes, s>>>(mk, mv, a, p.row_tiles, p.parts,
                                                                                    part);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join(a, p, part, s);
}

}  // namespace httm
