// Attention over key ranges for few query rows: single tokens, or a handful,
// against a long cache.  All query heads of a key head share K and V, so a
// work item is the R = q_len * group <= 32 rows of one key head.
//
// Bound by the memory K and V come from: a row's arithmetic hides behind its
// bytes, and a 128-row tensor-core tile would be mostly padding (the tiled
// kernel took 277 us where this one takes 169, 32 sequences of up to 41,070
// keys).  So every warp works alone: it streams tiles of 32 keys by TMA into
// a ring of its own (no barrier with another warp until the end), multiplies
// with the 16-row warp-level MMAs (m16n8k16), and keeps a running maximum,
// sum and O in fp32 registers (P enters P V in bf16, as in the tiled kernels).  Four warps a block and two blocks an SM keep about
// 128 KB of loads in flight.  At the end the block's warps are added up in
// order, then the blocks of an item: up to 8 are a cluster and read each
// other's shared memory (one launch, no workspace); more, for a long cache
// with few items, go through the workspace and attn_join_kernel.
#include <algorithm>

#include "attn_ops.cuh"

namespace httm {
namespace {

using namespace tc;

constexpr int kWarps = 4;
constexpr int kKeys = 32;                             // keys of a warp's tile
constexpr int kRing = 3;
constexpr uint32_t kHalf = kKeys * kAttnD * 2;        // 4 KB: 32 rows x 64 bf16 (K or V)
constexpr int kMaxRows = 32;
constexpr int kCluster = kAttnCluster;                // parts of an item that form a cluster

struct RowsSmem {
  uint8_t kv[kWarps][kRing][2][kHalf];                // reused for the warps' O at the end
  float m[kWarps][kMaxRows], l[kWarps][kMaxRows];
  float bm[kMaxRows], bl[kMaxRows];                   // the block's
  uint64_t full[kWarps][kRing];
  int abort;
};
constexpr size_t kRowsSmem = sizeof(RowsSmem) + 1024;
static_assert(kWarps * kMaxRows * kAttnD * 4 <= sizeof(RowsSmem::kv), "the warps' O fit the rings");
static_assert(2 * (kRowsSmem + 1024) <= 227 * 1024, "two blocks an SM");

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The address of a shared-memory location in block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_block(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Four channels of a finished row: O / l, and the log-sum-exp.
__device__ __forceinline__ void put_row(const AttnArgs& a, int b, int kh, int r, int c, float4 v, float mx, float l) {
  const int li = r / a.G, head = kh * a.G + (r - li * a.G);
  const int2 kr = key_range(a, b, li);
  const bool seen = kr.x < kr.y;
  const float inv = seen ? 1.f / l : 0.f;
  if (!seen) v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < a.d) {
    __nv_bfloat16* dst =
        reinterpret_cast<__nv_bfloat16*>(a.out.data) + b * a.out.sb + head * a.out.sh + (int64_t)li * a.out.st;
    *reinterpret_cast<uint2*>(dst + c) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
  }
  if (c == 0 && a.lse)
    a.lse[((size_t)b * a.H + head) * a.L + li] = seen ? (mx + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

// MT tiles of 16 rows.  CLUSTER: the parts of an item are one cluster.
template <int MT, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32, 2)
attn_rows_kernel(const __grid_constant__ AttnMap mk, const __grid_constant__ AttnMap mv,
                 const __grid_constant__ AttnArgs a, int parts, float* __restrict__ part_out) {
  extern __shared__ uint8_t smem_raw[];
  RowsSmem& sm = *reinterpret_cast<RowsSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned bk = blockIdx.x / parts, part = blockIdx.x % parts;
  const int b = bk / a.K, kh = bk % a.K, R = a.L * a.G;
  volatile int* abort = &sm.abort;
  DevState* st = a.st;

  // lane r: the keys of row r; the union of all rows' keys
  const int2 mine = lane < R ? key_range(a, b, lane / a.G) : make_int2(0, 0);
  const bool live = mine.x < mine.y;
  const int lo = warp_min(live ? mine.x : 0x7fffffff), hi = warp_max(live ? mine.y : 0);
  const int f_lo = warp_max(live ? mine.x : 0), f_hi = warp_min(live ? mine.y : 0x7fffffff);   // seen by all live rows
  const int n_all = lo < hi ? (hi - lo + kKeys - 1) / kKeys : 0;
  const int t0 = (int)((long long)n_all * part / parts), t1 = (int)((long long)n_all * (part + 1) / parts);
  const int n = t1 - t0 > warp ? (t1 - t0 - warp + kWarps - 1) / kWarps : 0;        // tiles of this warp
  auto first_key = [&](int i) { return lo + (t0 + warp + i * kWarps) * kKeys; };

  if (threadIdx.x == 0) sm.abort = 0;
  if (lane == 0)
    for (int s = 0; s < kRing; ++s) mbar_init(&sm.full[warp][s], 1);
  mbar_fence_init();
  __syncthreads();
  auto load = [&](int i) {
    uint64_t* bar = &sm.full[warp][i % kRing];
    mbar_arrive_expect_tx(bar, 2 * kHalf);
    tma_load_tile(sm.kv[warp][i % kRing][0], mk, bar, first_key(i), kh, b);
    tma_load_tile(sm.kv[warp][i % kRing][1], mv, bar, first_key(i), kh, b);
  };
  if (lane == 0)
    for (int i = 0; i < min(n, kRing); ++i) load(i);

  // Q as A fragments: lane holds rows lane / 4 and + 8, channel pairs 2 (lane % 4) and + 8
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  uint32_t q[MT][4][4];
  int2 keys[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = t * 16 + r0 + h * 8;
      const bool in = r < R;
      const int l = in ? r / a.G : 0, head = in ? kh * a.G + (r - l * a.G) : 0;
      const int2 kr = in ? key_range(a, b, l) : make_int2(0, 0);
      keys[t][h] = kr;
      const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(a.q.data) + b * a.q.sb + head * a.q.sh +
                                 (int64_t)l * a.q.st;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int c = kk * 16 + c0 + w * 8;
          q[t][kk][h + 2 * w] = kr.x < kr.y && c < a.d ? *reinterpret_cast<const uint32_t*>(src + c) : 0u;
        }
    }

  float o[MT][8][4], m[MT][2], sum[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    m[t][0] = m[t][1] = -INFINITY;
    sum[t][0] = sum[t][1] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][j][e] = 0.f;
  }

  bool ok = true;
  for (int i = 0; i < n; ++i) {
    const int s = i % kRing, k0 = first_key(i);
    if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[warp][s], (i / kRing) & 1, abort, st))) { ok = false; break; }
    uint8_t* ks = sm.kv[warp][s][0];
    uint8_t* vs = sm.kv[warp][s][1];
    if (hi - k0 < kKeys) {                            // V rows behind the union may hold anything
      zero_rows(vs, kKeys, [&](int r) { return r >= hi - k0; });
      __syncwarp();
    }
    const bool masked = k0 < f_lo || k0 + kKeys > f_hi;
    // a zero probability times an infinity or NaN is not zero: where a row
    // does not see the whole tile, such elements leave V (a row a lane) and
    // are added below to the rows that see them
    const bool mixed = k0 < f_lo || min(k0 + kKeys, hi) > f_hi;
    const uint32_t odd = mixed ? __ballot_sync(0xffffffffu, wild_row(vs, lane)) : 0u;
    if (odd >> lane & 1) {
      tame_row(vs, lane);
      fence_async_smem();                             // before the TMA load that reuses this stage
    }
    __syncwarp();
    const uint32_t ka = smem_u32(ks), va = smem_u32(vs);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      // S: 4 tiles of 8 keys
      float sc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
        const int row = j * 8 + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {              // 32 channels a load
          uint32_t x[4];
          ldsm4(ka + row * 128 + (((kk * 4 + (lane >> 3)) ^ (row & 7)) << 4), x);
          mma16(sc[j], q[t][2 * kk], x[0], x[1]);
          mma16(sc[j], q[t][2 * kk + 1], x[2], x[3]);
        }
      }
      if (masked) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = k0 + j * 8 + c0 + (e & 1);
            const int2 kr = keys[t][e >> 1];
            if (key < kr.x || key >= kr.y) sc[j][e] = -INFINITY;
          }
      }
      // running maximum and sum of rows r0 and r0 + 8
      float alpha[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = max3(mx, sc[j][2 * h], sc[j][2 * h + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(m[t][h], mx * a.scale_log2);
        const float ref = m_new == -INFINITY ? 0.f : m_new;      // nothing seen yet: P and the sum stay 0
        alpha[h] = ex2(m[t][h] - ref);
        m[t][h] = m_new;
        float x = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 2 * h; e < 2 * h + 2; ++e) {
            sc[j][e] = ex2(fmaf(sc[j][e], a.scale_log2, -ref));
            x += sc[j][e];
          }
        sum[t][h] = fmaf(sum[t][h], alpha[h], x);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[t][j][0] *= alpha[0], o[t][j][1] *= alpha[0];
          o[t][j][2] *= alpha[1], o[t][j][3] *= alpha[1];
        }
      }
      // O += P V: two steps of 16 keys
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const uint32_t p[4] = {pack_bf16(sc[2 * kk][0], sc[2 * kk][1]), pack_bf16(sc[2 * kk][2], sc[2 * kk][3]),
                               pack_bf16(sc[2 * kk + 1][0], sc[2 * kk + 1][1]),
                               pack_bf16(sc[2 * kk + 1][2], sc[2 * kk + 1][3])};
        const int row = kk * 16 + (lane & 15);        // matrices: keys 0-7, 8-15 of two 8-channel columns
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t x[4];
          ldsm4t(va + row * 128 + (((2 * j + (lane >> 4)) ^ (row & 7)) << 4), x);
          mma16(o[t][2 * j], p, x[0], x[1]);
          mma16(o[t][2 * j + 1], p, x[2], x[3]);
        }
      }
    }
    for (uint32_t rest = odd; rest; rest &= rest - 1) {
      const int key = k0 + __ffs(rest) - 1;
      const __nv_bfloat16* src =
          reinterpret_cast<const __nv_bfloat16*>(a.v.data) + b * a.v.sb + kh * a.v.sh + (int64_t)key * a.v.st;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = j * 8 + c0;
        if (key >= a.N || c >= a.d) continue;
        const uint32_t x = *reinterpret_cast<const uint32_t*>(src + c);
        if (!wild(x)) continue;
        const float v[2] = {__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)};
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int2 kr = keys[t][e >> 1];
            if (key >= kr.x && key < kr.y && !isfinite(v[e & 1])) o[t][j][e] += v[e & 1];
          }
      }
    }
    __syncwarp();
    if (lane == 0 && i + kRing < n) load(i + kRing);
  }
  if (!__syncthreads_and(ok)) {
    // a wait ran out: copies in flight land before the shared memory goes
    // away; the outputs are undefined, but every block meets the barriers
    for (int i = 0; i < 200; ++i) __nanosleep(1000);
  }

  // the warps' results, then their sum in order
  float* ow = reinterpret_cast<float*>(&sm.kv[0][0][0][0]) + warp * kMaxRows * kAttnD;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = t * 16 + r0 + h * 8;
      float x = sum[t][h];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      if ((lane & 3) == 0) {
        sm.m[warp][r] = m[t][h];
        sm.l[warp][r] = x;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float2*>(ow + r * kAttnD + j * 8 + c0) = make_float2(o[t][j][2 * h], o[t][j][2 * h + 1]);
    }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(&sm.kv[0][0][0][0]);
  for (int x = threadIdx.x; x < R * (kAttnD / 4); x += kWarps * 32) {
    const int r = x / (kAttnD / 4), c = (x % (kAttnD / 4)) * 4;
    float mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][r]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(sm.m[w][r] - ref);
      const float4 y = *reinterpret_cast<const float4*>(all + (w * kMaxRows + r) * kAttnD + c);
      l = fmaf(sm.l[w][r], f, l);
      v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
    }
    if (CLUSTER) {
      // over the first warp's O, which this thread alone reads here
      float* own = reinterpret_cast<float*>(&sm.kv[0][0][0][0]);
      *reinterpret_cast<float4*>(own + r * kAttnD + c) = v;
      if (c == 0) {
        sm.bm[r] = mx;
        sm.bl[r] = l;
      }
    } else if (parts > 1) {
      float* dst = part_out + ((size_t)blockIdx.x * R + r) * kAttnRangePart;
      *reinterpret_cast<float4*>(dst + c) = v;
      if (c == 0) {
        dst[kAttnD] = l;
        dst[kAttnD + 1] = mx;
      }
    } else {
      put_row(a, b, kh, r, c, v, mx, l);
    }
  }
  if (CLUSTER) {
    cluster_sync();
    // each block finishes its share of the rows, reading the others' in order
    for (int x = threadIdx.x; x < R * (kAttnD / 4); x += kWarps * 32) {
      const int r = x / (kAttnD / 4), c = (x % (kAttnD / 4)) * 4;
      if ((unsigned)r % parts != part) continue;
      float mx = -INFINITY, l = 0.f;
      for (int p = 0; p < parts; ++p) mx = fmaxf(mx, ld_cluster(in_block(&sm.bm[r], p)));
      const float ref = mx == -INFINITY ? 0.f : mx;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = 0; p < parts; ++p) {
        const float f = ex2(ld_cluster(in_block(&sm.bm[r], p)) - ref);
        const float4 y = ld_cluster4(in_block(all + r * kAttnD + c, p));
        l = fmaf(ld_cluster(in_block(&sm.bl[r], p)), f, l);
        v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
      }
      put_row(a, b, kh, r, c, v, mx, l);
    }
    cluster_sync();                                   // nobody leaves while its memory is read
  }
}

}  // namespace

// Parts of an item's keys: blocks stream about 128 keys (four warps' tiles)
// at a time, and cost about four such rounds of start and end; two are
// resident on an SM.  Where ranges are given the entries' lengths may differ,
// so the items are cut in enough parts to even out.  Up to kCluster parts
// cost little to add up (rounded to a power of two: clusters of other sizes
// leave SMs idle); beyond that the join is a launch of its own.
int attn_rows_parts(const httm_attention& a, bool ranges) {
  const long long items = (long long)a.batch * a.kv_heads, rounds = (a.kv_len + kWarps * kKeys - 1) / (kWarps * kKeys);
  const int slots = 2 * kSMs;
  const int most = (int)std::min<long long>(kAttnMaxParts, std::max<long long>(1, rounds));
  int parts = 1;
  double best = 0;
  for (int n = 1; n <= most && items > 0; ++n) {
    if (n <= kCluster && (n & (n - 1)) != 0) continue;
    if (n > 1 && items * n > 16 * slots) break;
    const long long waves = (items * n + slots - 1) / slots;
    double cost = (double)waves * ((rounds + n - 1) / n + 4) + (n > kCluster ? 4 + n / 8.0 : n > 1 ? 1 : 0);
    // ragged items: the longest part bounds the last wave
    if (ranges && waves < 4) cost += (double)(rounds + n - 1) / n * (4 - waves) / 4;
    if (best == 0 || cost < best) best = cost, parts = n;
  }
  return parts;
}

cudaError_t launch_attn_rows(const AttnArgs& a, const AttnFwdPlan& p, float* part_out, cudaStream_t s) {
  AttnMap mk, mv;
  // without keys nothing is loaded through their maps
  if (!attn_map(&mk, a.k, a.q.data, a.d, a.N, a.K, a.B, kKeys) || !attn_map(&mv, a.v, a.q.data, a.d, a.N, a.K, a.B, kKeys))
    return cudaErrorInvalidValue;
  const bool cluster = p.parts > 1 && p.parts <= kCluster;
  auto kernel = p.rows <= 16 ? (cluster ? attn_rows_kernel<1, true> : attn_rows_kernel<1, false>)
                             : (cluster ? attn_rows_kernel<2, true> : attn_rows_kernel<2, false>);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowsSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.items * p.parts));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kRowsSmem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim = {(unsigned)p.parts, 1, 1};
  cfg.attrs = &at;
  cfg.numAttrs = cluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, mk, mv, a, p.parts, part_out);
}

}  // namespace httm
