// Attention over key ranges, backward.  With P_ij = exp(c q_i.k_j - lse_i)
// recomputed from q, k and lse, and D_i = dout_i . out_i:
//   dV = P^T dO,  dP = dO V^T,  dS = P o (dP - D),  dQ = c dS K,  dK = c dS^T Q.
//
// Three launches (a fourth when key tiles are split):
//  - attn_prep_kernel: -D and -lse of every query row, padded to whole steps,
//    as fp32 and as operands of three bf16 (see below), and the key ranges of
//    rows and of steps;
//  - attn_dkv_kernel: a CTA owns 128 keys and walks over the query tiles
//    that see them, for all query heads sharing the key head; dK and dV stay
//    in TMEM.  Everything is transposed (rows = keys): S^T = K Q^T and dP^T
//    = V dO^T, so that P^T and dS^T are written back to TMEM as the A
//    operands of dV += P^T dO and dK += dS^T Q, and nothing passes through
//    shared memory but the loaded tiles;
//    Here lse and D belong to a column, not to a thread's row: reading them
//    from shared memory would cost 8 bytes an element of its bandwidth, as
//    much as all else together (dK/dV 1087 us).  Instead one more K step of
//    each product adds them: a row of ones times -lse / scale (-D) as the sum
//    of three bf16, which holds an fp32 whole (1023 us);
//  - attn_dq_kernel: a CTA owns 128 queries and walks over their keys; dS is
//    the A operand of dQ += dS K.
// Roundings: S, dP, the exponentials and the accumulators are fp32.  P and dS
// are rounded to bf16, at most 2^-8 of themselves, as operands of the tensor
// core beside bf16 dO, K and Q.  D comes from out as the forward left it, in
// bf16: an fp32 copy would be 4 more bytes an element to write and to read;
// D is off by 2^-8 sum |dout| |out| at most, which dS takes over times P.
// Over few keys, where P is large, that shows most.
//
// Seven products a tile where one fused pass has five: dQ gathered from
// key-owning CTAs needs either atomics, whose order would change the result
// from run to run, or N x N / 128 partial sums.
//
// Both kernels are made of groups: two warpgroups of 4 warps (TMEM lane =
// row, each with half of the columns) with an S and a dP of their own in
// TMEM, so that one group exponentiates while another forms dS and neither
// waits for the other's buffer.  P overwrites its S and dS its dP, as bf16
// pairs.  Short sequences run two blocks of one group an SM, long ones a
// block of two groups that take the even and the odd steps (Cfg).
// Warp 0 loads (TMA); one thread of warp 1 and one of warp 3 issue the MMAs:
// one alone issues an N = 64 product at half the tensor core's rate, two
// keep it fed.  They share the work so that a product which overwrites an
// operand is issued by the thread that issued that operand's use (the tensor
// core works in order of issue per thread), and so that every accumulator
// has one issuing thread: its order of summation is fixed.  For dK and dV
// warp 1 has S and dV, warp 3 dP and dK; for dQ each group has its issuing
// warp and an accumulator.  Warp 2 clears loaded rows that may hold anything.
//
// Parity waits: a barrier of a group completes one phase per step of that
// group, and no phase can begin before every waiter has seen the one before:
// S of the group's next step is issued behind the product that read P (or
// the reads of S), dP behind the product that read dS.
#include <algorithm>

#include "attn_ops.cuh"

namespace httm {
namespace {

using namespace tc;

// G groups a block (see above): 1 with two blocks an SM, 2 with one.
template <int G>
struct Cfg {
  static constexpr int kThreads = 128 + 256 * G, kBlocks = 3 - G;
  static constexpr uint32_t kTmem = 256 * G;          // tensor memory columns
  // registers a thread: launched at 80 or 96, then 128 kAuxRegs + 256 G
  // kWorkRegs of the same total
  static constexpr int kLaunchRegs = G == 1 ? 80 : 96, kAuxRegs = G == 1 ? 48 : 64, kWorkRegs = G == 1 ? 96 : 104;
  static constexpr int kRegs = 128 * kAuxRegs + 256 * G * kWorkRegs;
  static_assert(kRegs <= kThreads * kLaunchRegs, "registers");
  static_assert(kBlocks * kThreads * kLaunchRegs <= 65536, "registers");
  // dK, dV: queries of a step, columns of a thread, query tiles in flight
  static constexpr int kStep = G == 1 ? 64 : 96, kCols = kStep / 2, kStages = G == 1 ? 3 : 5;
  static constexpr uint32_t kStepBytes = kStep * kAttnD * 2;
  static constexpr uint32_t kColV = G * 2 * kStep, kColK = kColV + kAttnD;   // group g: S at 2 g kStep, dP kStep behind
  // dQ: the same for keys
  static constexpr int kKeyStep = 96, kKeyCols = kKeyStep / 2, kKvStages = 3 * G;
  static constexpr uint32_t kKeyBytes = kKeyStep * kAttnD * 2;
  static constexpr uint32_t kColQ = G * 2 * kKeyStep;                        // group g's dQ at kColQ + 64 g
  static_assert(kColK + kAttnD <= kTmem && kColQ + G * kAttnD <= kTmem, "tensor memory");
  static_assert(kStepBytes % 1024 == 0 && kKeyBytes % 1024 == 0, "tiles start on 1024 bytes");
};
constexpr int kMaxQTiles = kAttnMaxQ / 64;
constexpr int kMaxWords = kMaxQTiles / 32;
constexpr int kChunk = 16;                            // columns in registers at a time
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ prep
// x as the sum of three bf16 (24 bits: all of an fp32), and five zeros.
__device__ __forceinline__ uint4 three_bf16(float x) {
  const float hi = __bfloat162float(__float2bfloat16_rn(x)), mid = __bfloat162float(__float2bfloat16_rn(x - hi));
  return make_uint4(pack_bf16(hi, mid), pack_bf16(x - hi - mid, 0.f), 0u, 0u);
}

// One step's rows of one head a block, 8 threads a row.
template <int kStep>
__global__ void __launch_bounds__(256)
attn_prep_kernel(const __grid_constant__ AttnArgs a, int q_tiles, float* __restrict__ nlse, float* __restrict__ ndsum,
                 uint4* __restrict__ extra, int2* __restrict__ ranges, AttnTileRange* __restrict__ tiles) {
  __shared__ AttnTileRange part[8];
  const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H, c = threadIdx.x & 7;
  const size_t Lp = (size_t)q_tiles * kStep;
  AttnTileRange tr{0x7fffffff, 0, 0, 0x7fffffff, 0, {0, 0, 0}};
#pragma unroll
  for (int pass = 0; pass < kStep / 32; ++pass) {
    const int l = blockIdx.x * kStep + pass * 32 + (threadIdx.x >> 3);
    const int2 keys = l < a.L ? key_range(a, b, l) : make_int2(0, 0);
    const bool live = keys.x < keys.y;
    float s = 0.f;
    if (live && c * 8 < a.d) {
      const uint4 x = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.dout.data) +
                                                     b * a.dout.sb + h * a.dout.sh + l * a.dout.st)[c];
      const uint4 y = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.out.data) + b * a.out.sb +
                                                     h * a.out.sh + l * a.out.st)[c];
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), s);
        s = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), s);
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == 0) {
      const float lse = live ? a.lse_in[(size_t)bh * a.L + l] : 0.f;
      nlse[bh * Lp + l] = live ? lse * -kLog2e : -INFINITY;
      ndsum[bh * Lp + l] = -s;
      uint4* e = extra + ((size_t)bh * q_tiles + blockIdx.x) * 2 * kStep + (l - blockIdx.x * kStep);
      e[0] = three_bf16(lse * (-1.f / a.scale));
      e[kStep] = three_bf16(-s);
      if (h == 0) ranges[b * Lp + l] = keys;
    }
    if (live) {
      tr.lo = min(tr.lo, keys.x);
      tr.hi = max(tr.hi, keys.y);
      tr.flo = max(tr.flo, keys.x);
      tr.fhi = min(tr.fhi, keys.y);
    } else if (l < a.L && c == 0) {
      ++tr.dead;
    }
  }
  if (h != 0) return;
  tr.lo = warp_min(tr.lo);
  tr.hi = warp_max(tr.hi);
  tr.flo = warp_max(tr.flo);
  tr.fhi = warp_min(tr.fhi);
  tr.dead = __reduce_add_sync(0xffffffffu, tr.dead);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = tr;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) {
      tr.lo = min(tr.lo, part[w].lo);
      tr.hi = max(tr.hi, part[w].hi);
      tr.flo = max(tr.flo, part[w].flo);
      tr.fhi = min(tr.fhi, part[w].fhi);
      tr.dead += part[w].dead;
    }
    tiles[(size_t)b * q_tiles + blockIdx.x] = tr;
  }
}

// Descriptor of a tile; K steps only add to its address field (shared memory
// addresses in 16-byte units stay below the field's 14 bits).
__device__ __forceinline__ uint64_t tile_desc(const uint8_t* tile) { return sw128_desc(smem_u32(tile), 1024); }

// D (+)= A B^T: K-major tiles of 128 and of N rows x 64 channels.
template <int N>
__device__ __forceinline__ void mma_rows(uint32_t d, uint64_t A, uint64_t B, bool add) {
  constexpr uint32_t id = idesc_bf16(128, N, false, false);
#pragma unroll
  for (int kk = 0; kk < kAttnD / 16; ++kk) umma_bf16(d, A + kk * 2, B + kk * 2, id, (add || kk > 0) ? 1u : 0u);
}
// D (+)= A B: A the 128 x N P or dS that the two warpgroups wrote to the front
// of their halves of the product at `A`; B a tile of N rows x 64 channels.
template <int N>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t A, uint64_t B, bool add) {
  constexpr uint32_t id = idesc_bf16(128, kAttnD, false, true);
  constexpr int per = N / 32;                         // K steps of one warpgroup's columns
#pragma unroll
  for (int kk = 0; kk < N / 16; ++kk)
    umma_bf16_ts(d, A + (kk / per) * (N / 2) + (kk % per) * 8, B + kk * 128, id, (add || kk > 0) ? 1u : 0u);
}

// Two neighbouring scores: s -> 2^(s c + m), or 2^(s c).
__device__ __forceinline__ void exp2_pair(uint32_t& s0, uint32_t& s1, unsigned long long cc, unsigned long long m) {
  float x0, x1;
  f2_unpack(f2_fma(f2_pack(__uint_as_float(s0), __uint_as_float(s1)), cc, m), x0, x1);
  s0 = __float_as_uint(ex2(x0));
  s1 = __float_as_uint(ex2(x1));
}
__device__ __forceinline__ void exp2_pair(uint32_t& s0, uint32_t& s1, unsigned long long cc) {
  float x0, x1;
  f2_unpack(f2_mul(f2_pack(__uint_as_float(s0), __uint_as_float(s1)), cc), x0, x1);
  s0 = __float_as_uint(ex2(x0));
  s1 = __float_as_uint(ex2(x1));
}
// Two neighbouring products, packed to bf16.
__device__ __forceinline__ uint32_t mul_pair(uint32_t p0, uint32_t p1, uint32_t g0, uint32_t g1) {
  float x0, x1;
  f2_unpack(f2_mul(f2_pack(__uint_as_float(p0), __uint_as_float(p1)), f2_pack(__uint_as_float(g0), __uint_as_float(g1))),
            x0, x1);
  return pack_bf16(x0, x1);
}
// Two neighbouring p (dP + nd), packed to bf16.
__device__ __forceinline__ uint32_t ds_pair(uint32_t p0, uint32_t p1, uint32_t g0, uint32_t g1, unsigned long long nd) {
  float x0, x1;
  f2_unpack(f2_mul(f2_pack(__uint_as_float(p0), __uint_as_float(p1)),
                   f2_add(f2_pack(__uint_as_float(g0), __uint_as_float(g1)), nd)), x0, x1);
  return pack_bf16(x0, x1);
}

// ------------------------------------------------------------------ dK, dV
template <int G>
struct DkvSmem {
  static constexpr int kStages = Cfg<G>::kStages, kStep = Cfg<G>::kStep, kStepBytes = Cfg<G>::kStepBytes;
  uint8_t k[kTileBytes], v[kTileBytes];
  uint8_t q[kStages][kStepBytes], g[kStages][kStepBytes];     // query and dout tiles
  uint4 ones[2][kAttnTile];                                   // K = 16 operand: 1 1 1 0 0 0 0 0, and zeros
  uint4 extra[kStages][2][kStep];                             // its counterpart: -lse / scale, and -D
  uint4 zeros[kStep];                                         // and the counterpart's other 8 columns
  int2 range[kStages][kStep];
  int flags[kStages];                                         // kMasked, kDead of the step in each stage
  uint32_t active[kMaxWords], masked[kMaxWords], dead[kMaxWords];
  uint64_t kv_full, q_full[kStages], q_empty[kStages];
  uint64_t s_full[G], dp_full[G], p_ready[G], ds_ready[G], drain, dirty, clean;
  int count[Cfg<G>::kThreads / 32];
  uint32_t tmem_base;
  int abort;
};
constexpr int kMasked = 1, kDead = 2;
template <int G>
constexpr size_t kDkvSmem = sizeof(DkvSmem<G>) + 1024;
static_assert(2 * (kDkvSmem<1> + 1024) <= 227 * 1024 && kDkvSmem<2> <= 226 * 1024, "shared memory");

// Walks over the set bits of `active`, round after round (one per head).
struct TileWalk {
  const uint32_t* bits;
  int words, w;
  uint32_t cur;
  int head;
  __device__ TileWalk(const uint32_t* bits_, int words_, int n_active, int start)
      : bits(bits_), words(words_), w(0), cur(0), head(0) {
    if (n_active == 0) return;                                  // nothing to walk: next() is not called
    cur = bits[0];
    head = start / n_active;
    int skip = start % n_active;                                // below n_active: ends before the last set bit
    while (skip >= __popc(cur)) {
      skip -= __popc(cur);
      cur = bits[++w];
    }
    for (; skip > 0; --skip) cur &= cur - 1;
  }
  // the next tile (there is always one: the walk wraps to the next head)
  __device__ int next() {
    while (cur == 0) {
      if (++w == words) {
        w = 0;
        ++head;
      }
      cur = bits[w];
    }
    const int t = w * 32 + __ffs(cur) - 1;
    cur &= cur - 1;
    return t;
  }
};

template <int G>
__global__ void __launch_bounds__(Cfg<G>::kThreads, Cfg<G>::kBlocks)
attn_dkv_kernel(const __grid_constant__ AttnMap mq, const __grid_constant__ AttnMap mg,
                const __grid_constant__ AttnMap mk, const __grid_constant__ AttnMap mv,
                const __grid_constant__ AttnArgs a, int q_tiles, int k_tiles, int parts,
                const uint4* __restrict__ extra, const int2* __restrict__ ranges,
                const AttnTileRange* __restrict__ tiles, float* __restrict__ part_out) {
  using C = Cfg<G>;
  constexpr int kStep = C::kStep, kCols = C::kCols, kStages = C::kStages, kThreads = C::kThreads;
  constexpr uint32_t kStepBytes = C::kStepBytes;
  extern __shared__ uint8_t smem_raw[];
  DkvSmem<G>& sm = *reinterpret_cast<DkvSmem<G>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x / parts, part = blockIdx.x % parts;
  const int bk = item / k_tiles, kt = item % k_tiles, b = bk / a.K, kh = bk % a.K;
  const int k0 = kt * kAttnTile, k1 = min(k0 + kAttnTile, a.N);
  const int words = (q_tiles + 31) / 32;
  const size_t Lp = (size_t)q_tiles * kStep;
  DevState* st = a.st;

  // which query tiles see these keys, which of them need compares, which
  // hold rows that see nothing
  int mine = 0;
  for (int w = warp; w < words; w += kThreads / 32) {
    const int t = w * 32 + lane;
    bool act = false, msk = false, ded = false;
    if (t < q_tiles) {
      const AttnTileRange r = tiles[(size_t)b * q_tiles + t];
      act = r.lo < r.hi && r.lo < k1 && r.hi > k0;
      msk = !(r.flo <= k0 && r.fhi >= k1);
      ded = r.dead > 0;
    }
    const uint32_t wa = __ballot_sync(0xffffffffu, act), wm = __ballot_sync(0xffffffffu, msk),
                   wd = __ballot_sync(0xffffffffu, ded);
    if (lane == 0) {
      sm.active[w] = wa;
      sm.masked[w] = wm;
      sm.dead[w] = wd;
    }
    mine += __popc(wa);
  }
  if (lane == 0) sm.count[warp] = mine;
  for (int r = threadIdx.x; r < kAttnTile; r += kThreads) {
    sm.ones[0][r] = make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u);
    sm.ones[1][r] = make_uint4(0u, 0u, 0u, 0u);
    if (r < kStep) sm.zeros[r] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_async_smem();
  if (threadIdx.x == 0) {
    mbar_init(&sm.kv_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 2);
    }
    for (int g = 0; g < G; ++g) {
      mbar_init(&sm.s_full[g], 1);
      mbar_init(&sm.dp_full[g], 1);
      mbar_init(&sm.p_ready[g], 256);
      mbar_init(&sm.ds_ready[g], 256);
    }
    mbar_init(&sm.drain, 2);
    mbar_init(&sm.dirty, 2);
    mbar_init(&sm.clean, 1);
    sm.abort = 0;
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(&sm.tmem_base, C::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  int n_active = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) n_active += sm.count[w];
  const long long all = (long long)n_active * a.G;
  const int s0 = (int)(all * part / parts), n = uniform((int)(all * (part + 1) / parts) - s0);   // steps of this CTA

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kAuxRegs) : "memory");
    if (warp == 0 && lane == 0 && n > 0) {
      // ------------------------------------------------------------ producer
      mbar_arrive_expect_tx(&sm.kv_full, 2 * kTileBytes);
      tma_load_tile(sm.k, mk, &sm.kv_full, k0, kh, b);
      tma_load_tile(sm.v, mv, &sm.kv_full, k0, kh, b);
      TileWalk walk(sm.active, words, n_active, s0);
      for (int i = 0; i < n; ++i) {
        const int s = i % kStages, t = walk.next(), h = kh * a.G + walk.head;
        if (i >= kStages && !mbar_wait(&sm.q_empty[s], ((i / kStages) - 1) & 1, abort, st)) break;
        sm.flags[s] = (sm.masked[t >> 5] >> (t & 31) & 1) * kMasked + (sm.dead[t >> 5] >> (t & 31) & 1) * kDead;
        mbar_arrive_expect_tx(&sm.q_full[s], 2 * kStepBytes + kStep * 40);
        tma_load_tile(sm.q[s], mq, &sm.q_full[s], t * kStep, h, b);
        tma_load_tile(sm.g[s], mg, &sm.q_full[s], t * kStep, h, b);
        bulk_load(sm.extra[s], extra + (((size_t)b * a.H + h) * q_tiles + t) * 2 * kStep, kStep * 32, &sm.q_full[s]);
        bulk_load(sm.range[s], ranges + b * Lp + (size_t)t * kStep, kStep * 8, &sm.q_full[s]);
      }
    } else if ((warp == 1 || warp == 3) && n > 0) {
      // ------------------------------------------------------------ MMA issue
      // warp 1: S^T = K Q^T and dV += P^T dO; warp 3: dP^T = V dO^T and dK +=
      // dS^T Q.  A group's next S (dP) overwrites the P (dS) it follows.
      const bool first = warp == 1;
      const uint64_t own = tile_desc(first ? sm.k : sm.v);
      const uint64_t rows = tile_desc(first ? sm.q[0] : sm.g[0]), cols = tile_desc(first ? sm.g[0] : sm.q[0]);
      // one more K step adds -lse / scale to S and -D to dP
      constexpr uint32_t id = idesc_bf16(128, kStep, false, false);
      const uint64_t one = plain_desc(smem_u32(sm.ones), kAttnTile * 16, 128);
      const uint32_t ext0 = smem_u32(sm.extra[0][first ? 0 : 1]), zeros = smem_u32(sm.zeros);
      const uint32_t buf = tmem + (first ? 0 : kStep), acc = tmem + (first ? C::kColV : C::kColK);
      uint64_t* full = first ? sm.s_full : sm.dp_full;
      uint64_t* ready = first ? sm.p_ready : sm.ds_ready;
      int n_dirty = 0;
      // waits for the tiles of step i and clears rows that may hold anything
      auto loaded = [&](int i) -> bool {
        const int s = i % kStages;
        if (!wait_all(&sm.q_full[s], (i / kStages) & 1, abort, st)) return false;
        if (__any_sync(0xffffffffu, sm.flags[s] & kDead)) {
          if (lane == 0) mbar_arrive(&sm.dirty);
          if (!wait_all(&sm.clean, n_dirty++ & 1, abort, st)) return false;
        }
        return true;
      };
      // operands of product i (outside the elected branch: they stay uniform)
      auto row_desc = [&](int i) { return rows + (i % kStages) * (kStepBytes >> 4); };
      auto ext_desc = [&](int i) {
        const uint32_t ext = ext0 + (i % kStages) * (kStep * 32);
        return plain_desc(ext, zeros - ext, 128);
      };
      auto dest = [&](int i) { return buf + (i % G) * 2 * kStep; };
      bool ok = wait_all(&sm.kv_full, 0, abort, st);
      for (int i = 0; ok && i < min(G, n); ++i) {
        if (!(ok = loaded(i))) break;
        tc_fence_after();
        const uint64_t rd = row_desc(i), ed = ext_desc(i);
        const uint32_t d = dest(i);
        if (elect_one()) {
          umma_bf16(d, one, ed, id, 0u);
          mma_rows<kStep>(d, own, rd, true);
          umma_commit(&full[i % G]);
        }
        __syncwarp();
      }
      // what the next product needs is waited for first, so that it follows
      // the P (dS) it overwrites at once
      for (int i = 0; ok && i < n; ++i) {
        const int s = i % kStages, grp = i % G;
        const bool more = i + G < n;
        if (more && !loaded(i + G)) break;
        const uint64_t rd = row_desc(i + G), ed = ext_desc(i + G), cd = cols + s * (kStepBytes >> 4);
        const uint32_t d = dest(i);
        if (!wait_all(&ready[grp], (i / G) & 1, abort, st)) break;
        tc_fence_after();
        if (elect_one()) {
          mma_cols<kStep>(acc, d, cd, i > 0);
          umma_commit(&sm.q_empty[s]);
          if (more) {
            umma_bf16(d, one, ed, id, 0u);
            mma_rows<kStep>(d, own, rd, true);
            umma_commit(&full[grp]);
          }
        }
        __syncwarp();
      }
      if (elect_one()) {
        umma_commit(&sm.drain);                                 // every MMA ends before TMEM is released
        drain_mma(&sm.drain, 0);
      }
      __syncwarp();
    } else if (warp == 2 && n > 0) {
      // ------------------------------------------------------------ rows that see nothing
      TileWalk walk(sm.active, words, n_active, s0);
      int n_dirty = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i % kStages, t = walk.next();
        if (!(sm.dead[t >> 5] >> (t & 31) & 1)) continue;
        // both issuing threads say when they have reached the step, and wait
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.dirty, n_dirty++ & 1, abort, st)) ||
            !__all_sync(0xffffffffu, mbar_wait(&sm.q_full[s], (i / kStages) & 1, abort, st)))
          break;
        zero_rows(sm.q[s], kStep, [&](int r) { return sm.range[s][r].x >= sm.range[s][r].y; });
        zero_rows(sm.g[s], kStep, [&](int r) { return sm.range[s][r].x >= sm.range[s][r].y; });
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.clean);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kWorkRegs) : "memory");
    // ------------------------------------------------------------ P and dS
    const int wg = (warp - 4) >> 2, grp = wg >> 1, half = wg & 1, row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + grp * 2 * kStep + half * kCols, td = ts + kStep;
    const int key = k0 + row;
    const unsigned long long cc = f2_pack(a.scale_log2, a.scale_log2);
    bool ok = true;
    for (int i = grp; i < n; i += G) {
      const int s = i % kStages, m = i / G;
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.q_full[s], (i / kStages) & 1, abort, st)) ||
          !__all_sync(0xffffffffu, mbar_wait(&sm.s_full[grp], m & 1, abort, st))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool masked = __any_sync(0xffffffffu, sm.flags[s] & kMasked);
      // p = 2^(c (s - lse / scale)) of this key and the queries of the columns
      uint32_t p[kCols];
#pragma unroll
      for (int c = 0; c < kCols; c += kChunk) tmem_ld16(ts + c, *reinterpret_cast<uint32_t(*)[16]>(&p[c]));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < kCols / 2; ++e) exp2_pair(p[2 * e], p[2 * e + 1], cc);
      if (masked) {
        const int4* rp = reinterpret_cast<const int4*>(sm.range[s] + half * kCols);
#pragma unroll
        for (int e = 0; e < kCols / 2; ++e) {
          const int4 r = rp[e];
          if (key < r.x || key >= r.y) p[2 * e] = 0u;
          if (key < r.z || key >= r.w) p[2 * e + 1] = 0u;
        }
      }
#pragma unroll
      for (int c = 0; c < kCols; c += kChunk) {
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          pk[e] = pack_bf16(__uint_as_float(p[c + 2 * e]), __uint_as_float(p[c + 2 * e + 1]));
        tmem_st8(ts + c / 2, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.p_ready[grp]);
      // dS = P (dP - D)
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.dp_full[grp], m & 1, abort, st))) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kCols; c += kChunk) {
        uint32_t g[16], pk[8];
        tmem_ld16(td + c, g);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (p[c + e] == 0u) g[e] = 0u;                    // a value nobody sees may be NaN
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) pk[e] = mul_pair(p[c + 2 * e], p[c + 2 * e + 1], g[2 * e], g[2 * e + 1]);
        tmem_st8(td + c / 2, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.ds_ready[grp]);
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sm.drain, 0, abort, st));
    tc_fence_after();
    // the first half of the warpgroups store dV, the others dK
    if (ok) {
      constexpr int kOut = kAttnD / G;                          // channels of a warpgroup
      const int which = wg / G, o0 = wg % G * kOut;
      uint32_t o[kOut];
      if (n > 0) {
        const uint32_t src = tmem + lane_off + (which == 0 ? C::kColV : C::kColK) + o0;
#pragma unroll
        for (int c = 0; c < kOut; c += 32) tmem_ld32(src + c, *reinterpret_cast<uint32_t(*)[32]>(&o[c]));
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < kOut; ++e) o[e] = 0u;
      }
      if (parts > 1) {
        float4* dst =
            reinterpret_cast<float4*>(part_out + (((size_t)blockIdx.x * 2 + which) * kAttnTile + row) * kAttnD + o0);
#pragma unroll
        for (int v = 0; v < kOut / 4; ++v)
          dst[v] = make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]), __uint_as_float(o[4 * v + 2]),
                               __uint_as_float(o[4 * v + 3]));
      } else if (key < a.N) {
        const View& w = which == 0 ? a.dv : a.dk;
        __nv_bfloat16* dst =
            reinterpret_cast<__nv_bfloat16*>(w.data) + b * w.sb + kh * w.sh + (int64_t)key * w.st;
        store_row_bf16<kOut / 8>(o, dst, which == 0 ? 1.f : a.scale, o0, a.d);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (*abort)
      for (int i = 0; i < 200; ++i) __nanosleep(1000);           // copies in flight land
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Adds up the parts of split key tiles, in order: 8 threads a row, 8
// channels each.
__global__ void __launch_bounds__(256)
attn_dkv_join_kernel(const __grid_constant__ AttnArgs a, int k_tiles, int parts, const float* __restrict__ part_in) {
  const long long idx = (long long)blockIdx.x * 32 + (threadIdx.x >> 3);
  if (idx >= 2ll * a.B * a.K * a.N) return;
  const int c = threadIdx.x & 7, wg = (int)(idx & 1);
  const int key = (int)((idx >> 1) % a.N), bk = (int)((idx >> 1) / a.N);
  const long long item = (long long)bk * k_tiles + key / kAttnTile;
  const float* src =
      part_in + (((size_t)item * parts * 2 + wg) * kAttnTile + key % kAttnTile) * kAttnD + c * 8;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; ++p) {
    const float4* x = reinterpret_cast<const float4*>(src + (size_t)p * 2 * kAttnTile * kAttnD);
    const float4 u = x[0], v = x[1];
    o[0] += u.x, o[1] += u.y, o[2] += u.z, o[3] += u.w, o[4] += v.x, o[5] += v.y, o[6] += v.z, o[7] += v.w;
  }
  if (c * 8 >= a.d) return;
  const float f = wg == 0 ? 1.f : a.scale;
  const View& w = wg == 0 ? a.dv : a.dk;
  __nv_bfloat16* dst =
      reinterpret_cast<__nv_bfloat16*>(w.data) + bk / a.K * w.sb + bk % a.K * w.sh + (int64_t)key * w.st + c * 8;
  *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f),
                                              pack_bf16(o[4] * f, o[5] * f), pack_bf16(o[6] * f, o[7] * f));
}

// ------------------------------------------------------------------ dQ
template <int G>
struct DqSmem {
  static constexpr int kKvStages = Cfg<G>::kKvStages, kKeyBytes = Cfg<G>::kKeyBytes;
  uint8_t q[kTileBytes], g[kTileBytes];
  uint8_t k[kKvStages][kKeyBytes], v[kKvStages][kKeyBytes];
  uint64_t q_full, kv_full[kKvStages], kv_empty[kKvStages];
  uint64_t s_full[G], dp_full[G], s_read[G], ds_ready[G], drain, dirty, clean;
  alignas(16) int lo[4], hi[4], f_lo[4], f_hi[4];
  uint32_t tmem_base;
  int abort;
};
template <int G>
constexpr size_t kDqSmem = sizeof(DqSmem<G>) + 1024;
static_assert(2 * (kDqSmem<1> + 1024) <= 227 * 1024 && kDqSmem<2> <= 226 * 1024, "shared memory");

template <int G>
__global__ void __launch_bounds__(Cfg<G>::kThreads, Cfg<G>::kBlocks)
attn_dq_kernel(const __grid_constant__ AttnMap mq, const __grid_constant__ AttnMap mg,
               const __grid_constant__ AttnMap mk, const __grid_constant__ AttnMap mv,
               const __grid_constant__ AttnArgs a, int Lp, const float* __restrict__ nlse,
               const float* __restrict__ ndsum, const int2* __restrict__ ranges) {
  using C = Cfg<G>;
  constexpr int kKeyStep = C::kKeyStep, kKeyCols = C::kKeyCols, kKvStages = C::kKvStages;
  constexpr uint32_t kKeyBytes = C::kKeyBytes;
  extern __shared__ uint8_t smem_raw[];
  DqSmem<G>& sm = *reinterpret_cast<DqSmem<G>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int m_tiles = (a.L + kAttnTile - 1) / kAttnTile;        // tiles of 128 queries; later ones first
  const int bh = blockIdx.x / m_tiles, qt = m_tiles - 1 - blockIdx.x % m_tiles;
  const int b = bh / a.H, h = bh % a.H, kh = h / a.G;
  // this thread's query and its keys; the union of the tile's
  const int wg = (warp - 4) >> 2, grp = wg >> 1, half = wg & 1;
  const int row = (warp & 3) * 32 + lane, l = qt * kAttnTile + row;
  const int2 keys = warp >= 4 && l < a.L ? ranges[(size_t)b * Lp + l] : make_int2(0, 0);
  const bool live = keys.x < keys.y;
  if (warp >= 4 && warp < 8) {
    const int x = warp_min(live ? keys.x : 0x7fffffff), y = warp_max(live ? keys.y : 0);
    const int fx = warp_max(live ? keys.x : 0), fy = warp_min(live ? keys.y : 0x7fffffff);
    if (lane == 0) {
      sm.lo[warp - 4] = x;
      sm.hi[warp - 4] = y;
      sm.f_lo[warp - 4] = fx;
      sm.f_hi[warp - 4] = fy;
    }
  }
  DevState* st = a.st;

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < kKvStages; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    for (int g = 0; g < G; ++g) {
      mbar_init(&sm.s_full[g], 1);
      mbar_init(&sm.dp_full[g], 1);
      mbar_init(&sm.s_read[g], 256);
      mbar_init(&sm.ds_ready[g], 256);
    }
    mbar_init(&sm.drain, G);
    mbar_init(&sm.dirty, 1);
    mbar_init(&sm.clean, 1);
    sm.abort = 0;
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(&sm.tmem_base, C::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  const int lo = min(min(sm.lo[0], sm.lo[1]), min(sm.lo[2], sm.lo[3]));
  const int hi = max(max(sm.hi[0], sm.hi[1]), max(sm.hi[2], sm.hi[3]));
  const int n = uniform(lo < hi ? (hi - lo + kKeyStep - 1) / kKeyStep : 0), base = n > 0 ? lo : 0;
  const int n_last = hi - (base + (n - 1) * kKeyStep);             // keys of the union in the last step

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kAuxRegs) : "memory");
    if (warp == 0 && lane == 0 && n > 0) {
      // ------------------------------------------------------------ producer
      mbar_arrive_expect_tx(&sm.q_full, 2 * kTileBytes);
      tma_load_tile(sm.q, mq, &sm.q_full, qt * kAttnTile, h, b);
      tma_load_tile(sm.g, mg, &sm.q_full, qt * kAttnTile, h, b);
      for (int j = 0; j < n; ++j) {
        const int s = j % kKvStages;
        if (j >= kKvStages && !mbar_wait(&sm.kv_empty[s], ((j / kKvStages) - 1) & 1, abort, st)) break;
        mbar_arrive_expect_tx(&sm.kv_full[s], 2 * kKeyBytes);
        tma_load_tile(sm.k[s], mk, &sm.kv_full[s], base + j * kKeyStep, kh, b);
        tma_load_tile(sm.v[s], mv, &sm.kv_full[s], base + j * kKeyStep, kh, b);
      }
    } else if ((warp == 1 || (G == 2 && warp == 3)) && n > 0) {
      // ------------------------------------------------------------ MMA issue
      // a warp a group: S = Q K^T, dP = dO V^T, dQ_g += dS K
      const int g = warp >> 1;
      const uint64_t qd = tile_desc(sm.q), gd = tile_desc(sm.g), kd = tile_desc(sm.k[0]), vd = tile_desc(sm.v[0]);
      const uint32_t buf = tmem + g * 2 * kKeyStep, acc = tmem + C::kColQ + g * kAttnD;
      // waits for the tiles of step j; the last one's K rows behind the union are cleared
      auto loaded = [&](int j) -> bool {
        const int s = j % kKvStages;
        if (!wait_all(&sm.kv_full[s], (j / kKvStages) & 1, abort, st)) return false;
        if (j == n - 1 && n_last < kKeyStep) {
          if (lane == 0) mbar_arrive(&sm.dirty);
          if (!wait_all(&sm.clean, 0, abort, st)) return false;
        }
        return true;
      };
      bool ok = g < n && wait_all(&sm.q_full, 0, abort, st) && loaded(g);
      if (ok) {
        tc_fence_after();
        const uint64_t k1 = kd + g * (kKeyBytes >> 4), v1 = vd + g * (kKeyBytes >> 4);
        if (elect_one()) {
          mma_rows<kKeyStep>(buf, qd, k1, false);
          umma_commit(&sm.s_full[g]);
          mma_rows<kKeyStep>(buf + kKeyStep, gd, v1, false);
          umma_commit(&sm.dp_full[g]);
        }
        __syncwarp();
      }
      for (int j = g; ok && j < n; j += G) {
        const int m = j / G, s = j % kKvStages, s2 = (j + G) % kKvStages;
        const bool more = j + G < n;
        // operands outside the elected branches: they stay uniform
        const uint64_t k0 = kd + s * (kKeyBytes >> 4), k1 = kd + s2 * (kKeyBytes >> 4), v1 = vd + s2 * (kKeyBytes >> 4);
        if (more) {
          if (!wait_all(&sm.s_read[g], m & 1, abort, st) || !loaded(j + G)) break;
          tc_fence_after();
          if (elect_one()) {
            mma_rows<kKeyStep>(buf, qd, k1, false);
            umma_commit(&sm.s_full[g]);
          }
          __syncwarp();
        }
        if (!wait_all(&sm.ds_ready[g], m & 1, abort, st)) break;
        tc_fence_after();
        if (elect_one()) {
          mma_cols<kKeyStep>(acc, buf + kKeyStep, k0, m > 0);
          umma_commit(&sm.kv_empty[s]);
          if (more) {
            mma_rows<kKeyStep>(buf + kKeyStep, gd, v1, false);  // over the dS that dQ reads
            umma_commit(&sm.dp_full[g]);
          }
        }
        __syncwarp();
      }
      if (elect_one()) {
        umma_commit(&sm.drain);                                 // every MMA ends before TMEM is released
        drain_mma(&sm.drain, 0);
      }
      __syncwarp();
    } else if (warp == 2 && n > 0 && n_last < kKeyStep) {
      // ------------------------------------------------------------ K rows behind the union of the ranges
      const int s = (n - 1) % kKvStages;
      if (__all_sync(0xffffffffu, mbar_wait(&sm.dirty, 0, abort, st)) &&
          __all_sync(0xffffffffu, mbar_wait(&sm.kv_full[s], ((n - 1) / kKvStages) & 1, abort, st))) {
        zero_rows(sm.k[s], kKeyStep, [&](int r) { return r >= n_last; });
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.clean);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kWorkRegs) : "memory");
    // ------------------------------------------------------------ dS
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + grp * 2 * kKeyStep + half * kKeyCols, td = ts + kKeyStep;
    const float m2 = l < a.L ? nlse[(size_t)bh * Lp + l] : -INFINITY, nd = l < a.L ? ndsum[(size_t)bh * Lp + l] : 0.f;
    const int c0 = base + half * kKeyCols;                         // the key of this thread's first column in step 0
    const int f_lo = warp_max(live ? keys.x : 0) - c0;          // every live row of the warp sees [f_lo, f_hi)
    const int f_hi = warp_min(live ? keys.y : 0x7fffffff) - c0;
    const unsigned long long cc = f2_pack(a.scale_log2, a.scale_log2), mm = f2_pack(m2, m2), dd = f2_pack(nd, nd);
    bool ok = true;
    for (int j = grp; j < n; j += G) {
      const int m = j / G;
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[grp], m & 1, abort, st))) { ok = false; break; }
      tc_fence_after();
      uint32_t p[kKeyCols];
#pragma unroll
      for (int c = 0; c < kKeyCols; c += kChunk) tmem_ld16(ts + c, *reinterpret_cast<uint32_t(*)[16]>(&p[c]));
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&sm.s_read[grp]);
      // (read again each step: every live row of the tile sees [f_lo, f_hi))
      if (half == 0 && (max(max(sm.f_lo[0], sm.f_lo[1]), max(sm.f_lo[2], sm.f_lo[3])) > base + j * kKeyStep ||
                        min(min(sm.f_hi[0], sm.f_hi[1]), min(sm.f_hi[2], sm.f_hi[3])) < min(base + (j + 1) * kKeyStep, hi))) {
        // some row does not see all of this step, and its dS of 0 times an
        // infinity or NaN there would not be 0: S has read K as it is, so
        // rows that see such a key have their NaN in dS; dQ reads it without
        const int s = j % kKvStages;
        if (!wait_all(&sm.kv_full[s], (j / kKvStages) & 1, abort, st)) { ok = false; break; }
        if (row < kKeyStep && wild_row(sm.k[s], row)) {
          tame_row(sm.k[s], row);
          fence_async_smem();
        }
      }
      const bool masked = f_lo > j * kKeyStep || f_hi < j * kKeyStep + kKeyCols;
#pragma unroll
      for (int e = 0; e < kKeyCols / 2; ++e) exp2_pair(p[2 * e], p[2 * e + 1], cc, mm);
      if (masked) {
        const int first = keys.x - c0 - j * kKeyStep, last = keys.y - c0 - j * kKeyStep;
#pragma unroll
        for (int e = 0; e < kKeyCols; ++e)
          if (e < first || e >= last) p[e] = 0u;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.dp_full[grp], m & 1, abort, st))) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kKeyCols; c += kChunk) {
        uint32_t g[16], pk[8];
        tmem_ld16(td + c, g);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (p[c + e] == 0u) g[e] = 0u;                      // a value nobody sees may be NaN
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) pk[e] = ds_pair(p[c + 2 * e], p[c + 2 * e + 1], g[2 * e], g[2 * e + 1], dd);
        tmem_st8(td + c / 2, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.ds_ready[grp]);
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sm.drain, 0, abort, st));
    tc_fence_after();
    if (ok) {
      constexpr int kOut = kAttnD / (2 * G);                    // channels of a warpgroup
      const int o0 = wg * kOut;
      uint32_t o[kOut];
      auto sum_of = [&](int g, uint32_t (&x)[kOut]) {
#pragma unroll
        for (int c = 0; c < kOut; c += 16)
          tmem_ld16(tmem + lane_off + C::kColQ + g * kAttnD + o0 + c, *reinterpret_cast<uint32_t(*)[16]>(&x[c]));
        tmem_wait_ld();
      };
      if (n > 0) sum_of(0, o);
      if (G == 2 && n > 1) {                                    // the second group's sum
        uint32_t x[kOut];
        sum_of(1, x);
#pragma unroll
        for (int e = 0; e < kOut; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(x[e]));
      }
      if (n == 0 || !live) {
#pragma unroll
        for (int e = 0; e < kOut; ++e) o[e] = 0u;
      }
      if (l < a.L) {
        __nv_bfloat16* dst =
            reinterpret_cast<__nv_bfloat16*>(a.dq.data) + b * a.dq.sb + h * a.dq.sh + (int64_t)l * a.dq.st;
        store_row_bf16<kOut / 8>(o, dst, a.scale, o0, a.d);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (*abort)
      for (int i = 0; i < 200; ++i) __nanosleep(1000);           // copies in flight land
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Groups a block.  Two blocks of one group hide each other's start and end
// (about 7 us a block: setting up, the first loads and products, the drain);
// one block of two groups has longer steps and is faster once it has enough
// of them.  dK/dV at 16 heads: 8 x 1,369 tokens 170 us with two blocks, 178
// with one; 4 x 2,738 288 and 274; 8,214 593 and 515; 64 x 128 40 and 61.  dQ:
// 137 and 154; 223 and 228; 473 and 415; 37 and 54.
//
// Splits of a key tile's queries: as for the forward, waves of CTAs times
// their steps plus about three steps of start and end.
AttnBwdPlan attn_bwd_plan(const httm_attention& a) {
  AttnBwdPlan p{};
  const long long group = a.heads / a.kv_heads;
  p.kv_groups = group * a.q_len <= 16 * kAttnTile ? 1 : 2;
  p.q_groups = a.kv_len <= 22 * kAttnTile ? 1 : 2;
  p.step = p.kv_groups == 1 ? Cfg<1>::kStep : Cfg<2>::kStep;
  p.q_tiles = (a.q_len + p.step - 1) / p.step;
  p.k_tiles = (a.kv_len + kAttnTile - 1) / kAttnTile;
  p.Lp = p.q_tiles * p.step;
  const long long items = (long long)a.batch * a.kv_heads * p.k_tiles;
  const long long steps = group * p.q_tiles, slots = kSMs * (3 - p.kv_groups);
  p.kv_parts = 1;
  double best = 0;
  for (int n = 1; n <= std::min<long long>(16, std::max<long long>(1, steps)) && items > 0; ++n) {
    if (n > 1 && items * n > 4 * slots) break;
    const long long waves = (items * n + slots - 1) / slots;
    const double cost = (double)waves * ((steps + n - 1) / n + 3) + (n > 1 ? 4 + n / 4.0 : 0);
    if (n == 1 || cost < best) best = cost, p.kv_parts = n;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += up256(bytes);
    return o;
  };
  p.stat = take((size_t)2 * a.batch * a.heads * p.Lp * sizeof(float));
  p.extra = take((size_t)2 * a.batch * a.heads * p.Lp * 16);
  p.range = take((size_t)a.batch * p.Lp * sizeof(int2));
  p.tiles = take((size_t)a.batch * p.q_tiles * sizeof(AttnTileRange));
  p.part = take(p.kv_parts > 1 ? (size_t)items * p.kv_parts * 2 * kAttnTile * kAttnD * sizeof(float) : 0);
  p.total = off;
  return p;
}

namespace {

struct BwdBuffers {
  float *nlse, *ndsum, *part;
  uint4* extra;
  int2* ranges;
  AttnTileRange* tiles;
};

// With no queries (or no keys) nothing is loaded through their maps.
bool bwd_maps(const AttnArgs& a, int q_box, int kv_box, AttnMap (&m)[4]) {
  const void* any = a.L > 0 ? a.q.data : a.k.data;
  return attn_map(&m[0], a.q, any, a.d, a.L, a.H, a.B, q_box) && attn_map(&m[1], a.dout, any, a.d, a.L, a.H, a.B, q_box) &&
         attn_map(&m[2], a.k, any, a.d, a.N, a.K, a.B, kv_box) && attn_map(&m[3], a.v, any, a.d, a.N, a.K, a.B, kv_box);
}

template <int G>
cudaError_t launch_dkv(const AttnArgs& a, const AttnBwdPlan& p, const BwdBuffers& w, cudaStream_t s) {
  using C = Cfg<G>;
  cudaError_t e;
  if (p.q_tiles > 0) {
    attn_prep_kernel<C::kStep><<<dim3(p.q_tiles, a.B * a.H), 256, 0, s>>>(a, p.q_tiles, w.nlse, w.ndsum, w.extra,
                                                                         w.ranges, w.tiles);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (p.k_tiles == 0) return cudaSuccess;
  AttnMap m[4];
  if (!bwd_maps(a, C::kStep, kAttnTile, m)) return cudaErrorInvalidValue;
  e = check_registers<attn_dkv_kernel<G>>(C::kThreads, C::kRegs);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attn_dkv_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDkvSmem<G>);
  if (e != cudaSuccess) return e;
  const long long items = (long long)a.B * a.K * p.k_tiles;
  attn_dkv_kernel<G><<<(unsigned)(items * p.kv_parts), C::kThreads, kDkvSmem<G>, s>>>(
      m[0], m[1], m[2], m[3], a, p.q_tiles, p.k_tiles, p.kv_parts, w.extra, w.ranges, w.tiles, w.part);
  if ((e = cudaGetLastError()) != cudaSuccess || p.kv_parts == 1) return e;
  const long long rows = 2ll * a.B * a.K * a.N;
  attn_dkv_join_kernel<<<(unsigned)((rows + 31) / 32), 256, 0, s>>>(a, p.k_tiles, p.kv_parts, w.part);
  return cudaGetLastError();
}

template <int G>
cudaError_t launch_dq(const AttnArgs& a, const AttnBwdPlan& p, const BwdBuffers& w, cudaStream_t s) {
  using C = Cfg<G>;
  if (a.L == 0) return cudaSuccess;
  AttnMap m[4];
  if (!bwd_maps(a, kAttnTile, C::kKeyStep, m)) return cudaErrorInvalidValue;
  cudaError_t e = check_registers<attn_dq_kernel<G>>(C::kThreads, C::kRegs);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attn_dq_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDqSmem<G>);
  if (e != cudaSuccess) return e;
  const long long m_tiles = (a.L + kAttnTile - 1) / kAttnTile;
  attn_dq_kernel<G><<<(unsigned)(a.B * a.H * m_tiles), C::kThreads, kDqSmem<G>, s>>>(m[0], m[1], m[2], m[3], a, p.Lp,
                                                                                   w.nlse, w.ndsum, w.ranges);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnArgs& a, const AttnBwdPlan& p, void* ws, cudaStream_t s) {
  char* w = static_cast<char*>(ws);
  BwdBuffers buf;
  buf.nlse = reinterpret_cast<float*>(w + p.stat);
  buf.ndsum = buf.nlse + (size_t)a.B * a.H * p.Lp;
  buf.extra = reinterpret_cast<uint4*>(w + p.extra);
  buf.ranges = reinterpret_cast<int2*>(w + p.range);
  buf.tiles = reinterpret_cast<AttnTileRange*>(w + p.tiles);
  buf.part = reinterpret_cast<float*>(w + p.part);
  const cudaError_t e = p.kv_groups == 1 ? launch_dkv<1>(a, p, buf, s) : launch_dkv<2>(a, p, buf, s);
  if (e != cudaSuccess) return e;
  return p.q_groups == 1 ? launch_dq<1>(a, p, buf, s) : launch_dq<2>(a, p, buf, s);
}

}  // namespace httm
