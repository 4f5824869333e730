// The norms before and after a block, fused with its gate and residual:
//   y = rs * x + gate * Post(f)          (stored in the stream's type)
//   z = Pre(y as stored)                 (stored in the branch's type)
// and their gradients.  With n = (v - mean) * r the normalised row (mean = 0
// for RMSNorm) and u = dz * weight,
//   dv = r * (u - mean(u) - n * mean(u * n))      (no mean(u) for RMSNorm).
//
// Bound by memory: forward reads x and f once and writes y and z once (8
// bytes an element in bf16), backward reads dy, dz, f, y and writes dx, df
// (12 bytes).  A row stays in registers between its two norms; the mean is
// taken before the squares, so the variance does not cancel.
//
// Threads: a row belongs to NT threads, each with V vectors of 8 channels.
// Forward uses one warp a row up to 512 channels and two up to 1,024 (65 us
// at 41,070 x 1,024 bf16, one warp a row 72, four 81); rows that only single
// elements can be taken from have twice the threads (5,476 x 1,001 fp32
// stream: 17 us against 20).
// Backward keeps the sums of up to five parameter gradients in registers
// while a thread group walks over its rows, so it spreads a row over more
// threads; each group writes one row of partial sums, which a second kernel
// adds up in a fixed order (no atomics: the result does not depend on the
// schedule).
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "ops.h"

namespace httm {
namespace {

constexpr int kMaxChannels = 8192;
constexpr int kMaxGates = 1024;

struct NormArgs {
  const void *x, *f, *y, *dy, *dz;      // x: forward only
  void *y_out, *z, *dx, *df;
  int64_t sx, sf, sy, sz, sdy, sdz, sdx, sdf;
  const float *gate, *post_w, *post_b, *pre_w, *pre_b;
  float *stats, *partial;
  int64_t rows, gate_rows;              // rows sharing a gate row
  int C, gates;
  int post, pre;
  float post_eps, pre_eps, rs;
  int chunks;                           // backward: thread groups per gate group
  unsigned want;                        // backward: bit k = parameter gradient k is wanted
};
enum { kGate = 0, kPostW, kPostB, kPreW, kPreB, kNumGrads };

// W neighbouring elements, 1 to 8, as raw words: bf16 pairs (a single bf16 in
// the low half) or fp32.  Converted when they are used, so a row in flight
// costs few registers and nothing waits for it.
template <class T, int W>
struct Words {
  static constexpr int n = W * (int)sizeof(T) <= 4 ? 1 : W * (int)sizeof(T) / 4;
  uint32_t w[n];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < n; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (W * sizeof(T) == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (n == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (n == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < n / 4; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    return __uint_as_float((e & 1) ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < W; ++e) w[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], W == 1 ? 0.f : v[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (W * sizeof(T) == 2) {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    } else if constexpr (n == 1) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (n == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < n / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
};

// The channels of a thread: E of them at v, as E / W vectors of W neighbours.
// W is E where the channels are a multiple of 8 and every row starts on 16
// bytes, 2 where rows allow pairs, else 1; the vectors of a thread are NT
// apart, so that neighbouring threads touch neighbouring memory.
template <int NT, int W, int E = 8>
struct Cols {
  int t, C;
  __device__ __forceinline__ int at(int v, int e) const { return ((v * (E / W) + e / W) * NT + t) * W + e % W; }
  __device__ __forceinline__ bool live(int v, int e) const { return at(v, e / W * W) < C; }
  // elements behind the row's end read as 0
  template <class T>
  __device__ __forceinline__ void load(const T* row, int v, float (&r)[E]) const {
#pragma unroll
    for (int e = 0; e < E; e += W) {
      Words<T, W> w;
      w.clear();
      if (live(v, e)) w.load(row + at(v, e));
#pragma unroll
      for (int i = 0; i < W; ++i) r[e + i] = w.get(i);
    }
  }
  template <class T>
  __device__ __forceinline__ void store(T* row, int v, const float (&r)[E]) const {
#pragma unroll
    for (int e = 0; e < E; e += W)
      if (live(v, e)) {
        Words<T, W> w;
        w.set(r + e);
        w.store(row + at(v, e));
      }
  }
};

// A row's E channels of a thread as loaded.
template <class T, int NT, int W, int E>
struct Raw {
  Words<T, W> words[E / W];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < E / W; ++i) words[i].clear();
  }
  __device__ __forceinline__ void load(const Cols<NT, W, E>& cols, const void* base, int64_t row, int64_t stride) {
    const T* p = static_cast<const T*>(base) + row * stride;
#pragma unroll
    for (int e = 0; e < E; e += W)
      if (cols.live(0, e)) words[e / W].load(p + cols.at(0, e));
  }
  __device__ __forceinline__ void get(float (&v)[E]) const {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = words[e / W].get(e % W);
  }
};

// K sums (1 or 2) over the NT threads of a row; all of them get them.  Two
// share a warp's shuffles: the first exchange leaves one sum's terms to each
// half of the warp.  NT > 32 is one row a block: the warps' sums meet in
// `tmp` (used in turn, so one barrier is enough), where every thread adds
// them up itself, four a load, instead of by shuffles again (the gradients
// of 41,070 x 1,024 bf16: 121 -> 118 us).
template <int K>
using RowTmp = float[2][K][32];
template <int NT, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], RowTmp<K>& tmp, int& turn) {
  static_assert(K == 1 || K == 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool upper = lane & 16;
  float x = v[0];
  if constexpr (K == 2) {
    x = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], 16);
  } else {
    x += __shfl_xor_sync(0xffffffffu, x, 16);
  }
#pragma unroll
  for (int h = 8; h > 0; h >>= 1) x += __shfl_xor_sync(0xffffffffu, x, h);
  if constexpr (NT == 32) {
    v[0] = x;
    if constexpr (K == 2) {
      const float o = __shfl_xor_sync(0xffffffffu, x, 16);
      v[0] = upper ? o : x;
      v[1] = upper ? x : o;
    }
  } else {
    if (K == 2 ? (lane & 15) == 0 : lane == 0) tmp[turn][K == 2 ? lane >> 4 : 0][warp] = x;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float* t = tmp[turn][k];
      if constexpr (NT == 64) {
        v[k] = t[0] + t[1];
      } else {
        v[k] = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 128; ++i) {
          const float4 q = reinterpret_cast<const float4*>(t)[i];
          v[k] += (q.x + q.y) + (q.z + q.w);
        }
      }
    }
    turn ^= 1;
  }
}

// n = (v - mean) * r in place; returns mean and r.
template <int NT, int W, int V>
__device__ __forceinline__ void normalise(float (&v)[V][8], const Cols<NT, W>& cols, int kind, float eps, float inv_c,
                                          RowTmp<1>& tmp, int& turn, float& mean, float& r) {
  mean = 0.f;
  float s[1];
  if (kind == HTTM_NORM_LAYER) {
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[i][e];            // 0 behind the row's end
    row_sums<NT, 1>(s, tmp, turn);
    mean = s[0] * inv_c;
  }
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[i][e] = cols.live(i, e) ? v[i][e] - mean : 0.f;
      s[0] = fmaf(v[i][e], v[i][e], s[0]);
    }
  row_sums<NT, 1>(s, tmp, turn);
  r = rsqrtf(fmaf(s[0], inv_c, eps));
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= r;
}

template <int NT, int W, int V>
__device__ __forceinline__ void affine(float (&v)[V][8], const Cols<NT, W>& cols, const float* w, const float* b) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float g[8], o[8];
    if (w) {
      cols.load(w, i, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= g[e];
    }
    if (b) {
      cols.load(b, i, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += o[e];
    }
  }
}

template <class TX, class TF, int NT, int V, int W>
__global__ void __launch_bounds__(NT > 32 ? NT : 128) gated_norm_kernel(NormArgs a) {
  constexpr int kRows = NT > 32 ? 1 : 4;                      // rows per block (barriers need one)
  __shared__ __align__(16) RowTmp<1> tmp;
  int turn = 0;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
  if (row >= a.rows) return;                                  // whole warps: NT is a multiple of 32
  const Cols<NT, W> cols{(int)(threadIdx.x % NT), a.C};
  const float inv_c = 1.f / (float)a.C;
  float f[V][8], y[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) cols.load(static_cast<const TX*>(a.x) + row * a.sx, i, y[i]);
  if (a.f) {
#pragma unroll
    for (int i = 0; i < V; ++i) cols.load(static_cast<const TF*>(a.f) + row * a.sf, i, f[i]);
  }
  if (a.post != HTTM_NORM_NONE) {
    float mean, r;
    normalise<NT, W, V>(f, cols, a.post, a.post_eps, inv_c, tmp, turn, mean, r);
    if (a.stats && cols.t == 0) {
      a.stats[row] = mean;
      a.stats[a.rows + row] = r;
    }
    affine<NT, W, V>(f, cols, a.post_w, a.post_b);
  }
  if (a.gate) {
    const float* g = a.gate + (row / a.gate_rows) * a.C;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float gv[8];
      cols.load(g, i, gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] *= gv[e];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[i][e] = a.f ? fmaf(a.rs, y[i][e], f[i][e]) : a.rs * y[i][e];
      y[i][e] = to_f(from_f<TX>(y[i][e]));                    // the norm reads the stream as it is stored
    }
  if (a.y_out) {
#pragma unroll
    for (int i = 0; i < V; ++i) cols.store(static_cast<TX*>(a.y_out) + row * a.sy, i, y[i]);
  }
  if (a.pre != HTTM_NORM_NONE) {
    float mean, r;
    normalise<NT, W, V>(y, cols, a.pre, a.pre_eps, inv_c, tmp, turn, mean, r);
    if (a.stats && cols.t == 0) {
      a.stats[2 * a.rows + row] = mean;
      a.stats[3 * a.rows + row] = r;
    }
    affine<NT, W, V>(y, cols, a.pre_w, a.pre_b);
#pragma unroll
    for (int i = 0; i < V; ++i) cols.store(static_cast<TF*>(a.z) + row * a.sz, i, y[i]);
  }
}

// Backward: channels a thread, threads a row and blocks an SM.  The parameter
// sums and the row in flight are the registers: 8 channels a thread, or with
// five sums up to 2,048 channels 4, fit the 128 of 512 threads an SM (20,000
// rows, 8 against 4 channels: 1,024 bf16 47 and 52 us, 256 33 and 38, 2,048
// fp32 72 and 117; with five sums 1,024 fp32 134 and 82, 4,096 bf16 90 and
// 174).  More threads with fewer registers are no faster: 4 channels, five
// sums, 1,024 fp32 at 512 / 768 / 1,024 threads 82 / 107 / 140.  At over
// 4,096 channels a row takes 1,024 threads, and registers spill: 8,192 bf16
// 104 us, with five sums 186.
constexpr int grad_channels(int C, bool post) { return post && C <= 2048 ? 4 : 8; }
constexpr int grad_threads(int C, int E) {
  int nt = 32;
  while (nt * E < C) nt *= 2;
  return nt;
}
constexpr int grad_blocks(int NT) { return NT == 1024 ? 1 : 512 / (NT > 32 ? NT : 128); }

// Backward: thread group g of gate group q walks over its share of that
// group's rows with E channels a thread, one row ahead with its loads.  POST:
// there is a norm on the block's output (two more parameter gradients and
// another pair of sums a row).
template <class TX, class TF, int NT, int W, bool POST, int E>
__global__ void __launch_bounds__(NT > 32 ? NT : 128, grad_blocks(NT))
gated_norm_grad_kernel(NormArgs a) {
  constexpr int kGroups = NT > 32 ? 1 : 4;                    // thread groups per block (barriers need one)
  __shared__ __align__(16) RowTmp<2> tmp;
  int turn = 0;
  const int64_t group = (int64_t)blockIdx.x * kGroups + threadIdx.x / NT;
  const int n_gates = max(1, a.gates);
  if (group >= (int64_t)n_gates * a.chunks) return;
  const Cols<NT, W, E> cols{(int)(threadIdx.x % NT), a.C};
  const float inv_c = 1.f / (float)a.C;
  const int gq = (int)(group / a.chunks), chunk = (int)(group % a.chunks);
  const int64_t r0 = gq * a.gate_rows + a.gate_rows * chunk / a.chunks;
  const int64_t r1 = gq * a.gate_rows + a.gate_rows * (chunk + 1) / a.chunks;
  const bool pre = a.pre != HTTM_NORM_NONE;

  float gate[E], pre_w[E], post_w[POST ? E : 1], post_b[POST ? E : 1];
#pragma unroll
  for (int e = 0; e < E; ++e) gate[e] = pre_w[e] = 1.f;
  if (a.gate) cols.load(a.gate + (int64_t)gq * a.C, 0, gate);
  if (a.pre_w) cols.load(a.pre_w, 0, pre_w);
  if constexpr (POST) {
#pragma unroll
    for (int e = 0; e < E; ++e) post_w[e] = 1.f, post_b[e] = 0.f;
    if (a.post_w) cols.load(a.post_w, 0, post_w);
    if (a.post_b) cols.load(a.post_b, 0, post_b);
  }
  constexpr int kAcc = POST ? 5 : 3;
  enum { aGate = 0, aPreW, aPreB, aPostW, aPostB };
  float acc[kAcc][E];
#pragma unroll
  for (int k = 0; k < kAcc; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[k][e] = 0.f;

  Raw<TX, NT, W, E> next_dy, next_y;
  Raw<TF, NT, W, E> next_f, next_dz;
  next_dy.clear();
  next_y.clear();
  next_f.clear();
  next_dz.clear();
  float pre_mean = 0.f, pre_r = 0.f, post_mean = 0.f, post_r = 0.f;
  auto fetch = [&](int64_t row) {
    if (a.dy) next_dy.load(cols, a.dy, row, a.sdy);
    if (a.f) next_f.load(cols, a.f, row, a.sf);
    if (pre) {
      next_y.load(cols, a.y, row, a.sy);
      next_dz.load(cols, a.dz, row, a.sdz);
      pre_mean = a.pre == HTTM_NORM_LAYER ? a.stats[2 * a.rows + row] : 0.f;
      pre_r = a.stats[3 * a.rows + row];
    }
    if constexpr (POST) {
      post_mean = a.post == HTTM_NORM_LAYER ? a.stats[row] : 0.f;
      post_r = a.stats[a.rows + row];
    }
  };
  if (r0 < r1) fetch(r0);
  for (int64_t row = r0; row < r1; ++row) {
    float g[E], f[E], y[E], dz[E];
    next_dy.get(g);
    next_f.get(f);
    next_y.get(y);
    next_dz.get(dz);
    const float m_pre = pre_mean, r_pre = pre_r, m_post = post_mean, r_post = post_r;
    if (row + 1 < r1) fetch(row + 1);
    if (pre) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        y[e] = cols.live(0, e) ? (y[e] - m_pre) * r_pre : 0.f;
        acc[aPreW][e] = fmaf(dz[e], y[e], acc[aPreW][e]);
        acc[aPreB][e] += dz[e];
        dz[e] *= pre_w[e];
        s[0] += dz[e];
        s[1] = fmaf(dz[e], y[e], s[1]);
      }
      row_sums<NT, 2>(s, tmp, turn);
      const float m0 = a.pre == HTTM_NORM_LAYER ? s[0] * inv_c : 0.f, m1 = s[1] * inv_c;
#pragma unroll
      for (int e = 0; e < E; ++e)                             // (behind the row's end: 0, not -m0)
        g[e] = cols.live(0, e) ? fmaf(r_pre, dz[e] - m0 - y[e] * m1, g[e]) : 0.f;
    }
    if (a.dx) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = a.rs * g[e];
      cols.store(static_cast<TX*>(a.dx) + row * a.sdx, 0, o);
    }
    if (a.f) {
      if constexpr (!POST) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          acc[aGate][e] = fmaf(g[e], f[e], acc[aGate][e]);
          g[e] *= gate[e];
        }
      } else {
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          f[e] = cols.live(0, e) ? (f[e] - m_post) * r_post : 0.f;
          acc[aGate][e] = fmaf(g[e], fmaf(f[e], post_w[e], post_b[e]), acc[aGate][e]);
          g[e] *= gate[e];
          acc[aPostW][e] = fmaf(g[e], f[e], acc[aPostW][e]);
          acc[aPostB][e] += g[e];
          g[e] *= post_w[e];
          s[0] += g[e];
          s[1] = fmaf(g[e], f[e], s[1]);
        }
        row_sums<NT, 2>(s, tmp, turn);
        const float m0 = a.post == HTTM_NORM_LAYER ? s[0] * inv_c : 0.f, m1 = s[1] * inv_c;
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = r_post * (g[e] - m0 - f[e] * m1);
      }
      if (a.df) cols.store(static_cast<TF*>(a.df) + row * a.sdf, 0, g);
    }
  }
  // partial sums in the order of kGate .. kPreB, wanted ones only
  const int64_t n_part = (int64_t)n_gates * a.chunks;
  auto put = [&](int k, const float (&v)[E]) {
    if (a.want >> k & 1) cols.store(a.partial + ((int64_t)__popc(a.want & ((1u << k) - 1)) * n_part + group) * a.C, 0, v);
  };
  put(kGate, acc[aGate]);
  put(kPreW, acc[aPreW]);
  put(kPreB, acc[aPreB]);
  if constexpr (POST) {
    put(kPostW, acc[aPostW]);
    put(kPostB, acc[aPostB]);
  }
}

struct SumArgs {
  const float* partial;
  float* out[kNumGrads];     // wanted gradients, in the order of the partial sums
  int is_gate0;              // out[0] is the gate's: summed per gate group
  int C, gates, chunks;
};

// Adds up the partial rows: 16 channels a block, 64 threads down the rows,
// each in order, then the 64 in a fixed tree.
__global__ void __launch_bounds__(1024) norm_sum_kernel(SumArgs a) {
  __shared__ float s[64][17];
  // blockIdx.y: the gate rows first (if wanted), then the other gradients
  const int y = blockIdx.y, col = blockIdx.x * 16 + threadIdx.x;
  const bool per_gate = a.is_gate0 && y < a.gates;
  const int k = per_gate ? 0 : a.is_gate0 ? y - a.gates + 1 : y, gate = per_gate ? y : 0;
  const int64_t n_part = (int64_t)a.gates * a.chunks;
  const int64_t p0 = (int64_t)gate * a.chunks, n = per_gate ? a.chunks : n_part;
  float v = 0.f;
  if (col < a.C) {
    const float* p = a.partial + ((int64_t)k * n_part + p0) * a.C + col;
    for (int64_t i = threadIdx.y; i < n; i += 64 * 8) {       // 8 loads in flight
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = i + u * 64 < n ? p[(i + u * 64) * a.C] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) v += x[u];
    }
  }
  s[threadIdx.y][threadIdx.x] = v;
  for (int h = 32; h > 0; h >>= 1) {
    __syncthreads();
    if ((int)threadIdx.y < h) s[threadIdx.y][threadIdx.x] += s[threadIdx.y + h][threadIdx.x];
  }
  if (threadIdx.y == 0 && col < a.C)
    a.out[k][(int64_t)gate * a.C + col] = s[0][threadIdx.x];
}

// Thread groups per gate group of the backward kernel: as many as the SMs
// hold at once, at least 4 rows a group.
int grad_chunks(const httm_norm_cfg& c) {
  const int64_t gates = std::max(1, c.gates), rows = c.rows / gates;
  const int nt = grad_threads(c.channels, grad_channels(c.channels, c.post != HTTM_NORM_NONE));
  const int64_t want = std::max<int64_t>(1, kSMs * grad_blocks(nt) * (nt > 32 ? 1 : 4) / gates);
  return (int)std::max<int64_t>(1, std::min(want, rows / 4));
}

template <class TX, class TF, int W>
cudaError_t launch_forward(const NormArgs& a, cudaStream_t s) {
#define HTTM_NORM_FWD(NT, V)                                                                        \
  do {                                                                                              \
    constexpr int kRows = (NT) > 32 ? 1 : 4;                                                        \
    const int64_t grid = (a.rows + kRows - 1) / kRows;                                              \
    gated_norm_kernel<TX, TF, NT, V, W><<<(unsigned)grid, (NT) > 32 ? (NT) : 128, 0, s>>>(a);     \
  } while (0)
  if (W == 1 && a.C > 512) {
    if (a.C <= 1024) HTTM_NORM_FWD(128, 1);
    else if (a.C <= 2048) HTTM_NORM_FWD(256, 1);
    else if (a.C <= 4096) HTTM_NORM_FWD(512, 1);
    else HTTM_NORM_FWD(1024, 1);
  } else if (a.C <= 256) HTTM_NORM_FWD(32, 1);
  else if (a.C <= 512) HTTM_NORM_FWD(32, 2);
  else if (a.C <= 1024) HTTM_NORM_FWD(64, 2);
  else if (a.C <= 2048) HTTM_NORM_FWD(128, 2);
  else if (a.C <= 4096) HTTM_NORM_FWD(256, 2);
  else HTTM_NORM_FWD(512, 2);
#undef HTTM_NORM_FWD
  return cudaGetLastError();
}

template <class TX, class TF, int W, bool POST>
cudaError_t launch_grad(const NormArgs& a, cudaStream_t s) {
#define HTTM_NORM_BWD(NT, E)                                                                          \
  do {                                                                                                \
    constexpr int kGroups = (NT) > 32 ? 1 : 4;                                                        \
    const int64_t grid = ((int64_t)std::max(1, a.gates) * a.chunks + kGroups - 1) / kGroups;          \
    gated_norm_grad_kernel<TX, TF, NT, (W < E ? W : E), POST, E><<<(unsigned)grid, (NT) > 32 ? (NT) : 128, 0, s>>>(a); \
  } while (0)
  constexpr int E = POST ? 4 : 8;
  switch (grad_channels(a.C, POST) == E ? grad_threads(a.C, E) : 0) {
    case 32: HTTM_NORM_BWD(32, E); break;
    case 64: HTTM_NORM_BWD(64, E); break;
    case 128: HTTM_NORM_BWD(128, E); break;
    case 256: HTTM_NORM_BWD(256, E); break;
    case 512: HTTM_NORM_BWD(512, E); break;
    default:
      if (a.C <= 4096) HTTM_NORM_BWD(512, 8);
      else HTTM_NORM_BWD(1024, 8);
  }
#undef HTTM_NORM_BWD
  return cudaGetLastError();
}

httm_status check_cfg(const httm_norm_cfg* c) {
  if (!c) return HTTM_ERR_ARG;
  auto dtype_ok = [](int t) { return t == HTTM_BF16 || t == HTTM_F32; };
  if (c->rows < 0 || c->channels < 1 || c->gates < 0) return HTTM_ERR_ARG;
  if (!dtype_ok(c->stream_dtype) || !dtype_ok(c->branch_dtype)) return HTTM_ERR_ARG;
  for (int kind : {c->post, c->pre})
    if (kind < HTTM_NORM_NONE || kind > HTTM_NORM_RMS) return HTTM_ERR_ARG;
  if (c->gates > 0 && c->rows % c->gates != 0) return HTTM_ERR_ARG;
  if (!(c->post_eps >= 0.f) || !(c->pre_eps >= 0.f)) return HTTM_ERR_ARG;
  if (!(c->residual_scale - c->residual_scale == 0.f)) return HTTM_ERR_ARG;
  if (c->channels > kMaxChannels || c->gates > kMaxGates || c->rows > 0x7fffffffll) return HTTM_ERR_UNSUPPORTED;
  if (c->stream_dtype == HTTM_BF16 && c->branch_dtype == HTTM_F32) return HTTM_ERR_UNSUPPORTED;
  return HTTM_OK;
}

size_t elem(int dtype) { return dtype == HTTM_F32 ? 4 : 2; }

// A [rows, C] argument: present, aligned to its type, and (an output) with
// rows that do not overlap.  Narrows *width to the elements (8, 2 or 1) that
// all accesses can take at a time.
httm_status check_rows(const httm_rows* r, int64_t rows, int C, int dtype, bool output, int* width) {
  if (!r->data) return HTTM_ERR_ARG;
  if (!aligned(r->data, elem(dtype))) return HTTM_ERR_ALIGN;
  if (output && rows > 1 && (r->row < 0 ? -r->row : r->row) < C) return HTTM_ERR_ARG;
  const int64_t row = rows > 1 ? r->row : 0;
  if (!aligned(r->data, 16) || row % (int64_t)(16 / elem(dtype)) != 0) *width = std::min(*width, 2);
  if (!aligned(r->data, 2 * elem(dtype)) || row % 2 != 0) *width = 1;
  return HTTM_OK;
}
httm_status check_param(const float* p, int* width) {
  if (!p) return HTTM_OK;
  if (!aligned(p, 4)) return HTTM_ERR_ALIGN;
  if (!aligned(p, 16)) *width = std::min(*width, 2);
  if (!aligned(p, 8)) *width = 1;
  return HTTM_OK;
}
int row_width(int C) { return C % 8 == 0 ? 8 : C % 2 == 0 ? 2 : 1; }

template <class TX, class TF, class Fn>
cudaError_t by_width(int width, Fn&& fn) {
  if (width == 8) return fn(TX{}, TF{}, std::integral_constant<int, 8>{});
  if (width == 2) return fn(TX{}, TF{}, std::integral_constant<int, 2>{});
  return fn(TX{}, TF{}, std::integral_constant<int, 1>{});
}
template <class Fn>
cudaError_t by_type(const httm_norm_cfg& c, int width, Fn&& fn) {
  using bf16 = __nv_bfloat16;
  if (c.branch_dtype == HTTM_F32) return by_width<float, float>(width, fn);
  if (c.stream_dtype == HTTM_F32) return by_width<float, bf16>(width, fn);
  return by_width<bf16, bf16>(width, fn);
}

}  // namespace
}  // namespace httm

using namespace httm;

extern "C" {

httm_status httm_gated_norm_forward(const httm_norm_cfg* c, const httm_norm_weights* w, const httm_rows* x,
                                    const httm_rows* f, const httm_rows* y, const httm_rows* z, float* stats,
                                    void* stream) {
  HTTM_TRY(check_cfg(c));
  if (!w || !x || (c->pre != HTTM_NORM_NONE) != (z != nullptr)) return HTTM_ERR_ARG;
  if ((c->gates > 0) != (w->gate != nullptr)) return HTTM_ERR_ARG;
  if (!f && (c->post != HTTM_NORM_NONE || c->gates > 0)) return HTTM_ERR_ARG;
  if (!y && (f || c->residual_scale != 1.f || !z)) return HTTM_ERR_ARG;
  if (c->rows == 0) return HTTM_OK;
  int wide = row_width(c->channels);   // elements an access takes
  NormArgs a{};
  HTTM_TRY(check_rows(x, c->rows, c->channels, c->stream_dtype, false, &wide));
  a.x = x->data, a.sx = x->row;
  if (f) {
    HTTM_TRY(check_rows(f, c->rows, c->channels, c->branch_dtype, false, &wide));
    a.f = f->data, a.sf = f->row;
  }
  if (y) {
    HTTM_TRY(check_rows(y, c->rows, c->channels, c->stream_dtype, true, &wide));
    a.y_out = y->data, a.sy = y->row;
  }
  if (z) {
    HTTM_TRY(check_rows(z, c->rows, c->channels, c->branch_dtype, true, &wide));
    a.z = z->data, a.sz = z->row;
  }
  for (const float* p : {w->gate, w->post_weight, w->post_bias, w->pre_weight, w->pre_bias})
    HTTM_TRY(check_param(p, &wide));
  if (stats && !aligned(stats, 4)) return HTTM_ERR_ALIGN;
  a.gate = w->gate;
  a.post_w = w->post_weight, a.post_b = w->post_bias, a.pre_w = w->pre_weight, a.pre_b = w->pre_bias;
  a.stats = stats;
  a.rows = c->rows;
  a.gates = c->gates;
  a.gate_rows = c->rows / std::max(1, c->gates);
  a.C = c->channels;
  a.post = c->post, a.pre = c->pre;
  a.post_eps = c->post_eps, a.pre_eps = c->pre_eps, a.rs = c->residual_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  HTTM_OPS_LAUNCH(by_type(*c, wide, [&](auto tx, auto tf, auto width) {
    return launch_forward<decltype(tx), decltype(tf), decltype(width)::value>(a, s);
  }), s);
  return HTTM_OK;
}

httm_status httm_gated_norm_workspace_bytes(const httm_norm_cfg* c, size_t* bytes) {
  HTTM_TRY(check_cfg(c));
  if (!bytes) return HTTM_ERR_ARG;
  *bytes = (size_t)kNumGrads * std::max(1, c->gates) * grad_chunks(*c) * c->channels * sizeof(float);
  return HTTM_OK;
}

httm_status httm_gated_norm_backward(const httm_norm_cfg* c, const httm_norm_weights* w, const httm_rows* dy,
                                     const httm_rows* dz, const httm_rows* f, const httm_rows* y, const float* stats,
                                     const httm_rows* dx, const httm_rows* df, const httm_norm_grads* grads,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  HTTM_TRY(check_cfg(c));
  const bool pre = c->pre != HTTM_NORM_NONE, post = c->post != HTTM_NORM_NONE;
  if (!w || !grads || pre != (dz != nullptr)) return HTTM_ERR_ARG;
  if ((c->gates > 0) != (w->gate != nullptr)) return HTTM_ERR_ARG;
  if (!f && (post || c->gates > 0 || df)) return HTTM_ERR_ARG;
  if (pre && c->rows > 0 && !y) return HTTM_ERR_ARG;
  if ((pre || post) && c->rows > 0 && !stats) return HTTM_ERR_ARG;
  if ((grads->gate && !c->gates) || ((grads->post_weight || grads->post_bias) && !post) ||
      ((grads->pre_weight || grads->pre_bias) && !pre))
    return HTTM_ERR_ARG;
  int wide = row_width(c->channels);   // elements an access takes
  NormArgs a{};
  if (c->rows > 0) {
    if (dy) {
      HTTM_TRY(check_rows(dy, c->rows, c->channels, c->stream_dtype, false, &wide));
      a.dy = dy->data, a.sdy = dy->row;
    }
    if (dz) {
      HTTM_TRY(check_rows(dz, c->rows, c->channels, c->branch_dtype, false, &wide));
      a.dz = dz->data, a.sdz = dz->row;
    }
    if (f) {
      HTTM_TRY(check_rows(f, c->rows, c->channels, c->branch_dtype, false, &wide));
      a.f = f->data, a.sf = f->row;
    }
    if (pre) {
      HTTM_TRY(check_rows(y, c->rows, c->channels, c->stream_dtype, false, &wide));
      a.y = y->data, a.sy = y->row;
    }
    if (dx) {
      HTTM_TRY(check_rows(dx, c->rows, c->channels, c->stream_dtype, true, &wide));
      a.dx = dx->data, a.sdx = dx->row;
    }
    if (df) {
      HTTM_TRY(check_rows(df, c->rows, c->channels, c->branch_dtype, true, &wide));
      a.df = df->data, a.sdf = df->row;
    }
  }
  for (const float* p : {w->gate, w->post_weight, w->post_bias, w->pre_weight, w->pre_bias})
    HTTM_TRY(check_param(p, &wide));
  int any = 8;
  for (const float* p : {grads->gate, grads->post_weight, grads->post_bias, grads->pre_weight, grads->pre_bias})
    HTTM_TRY(check_param(p, &any));
  if (stats && !aligned(stats, 4)) return HTTM_ERR_ALIGN;
  SumArgs sum{};
  float* outs[kNumGrads] = {grads->gate, grads->post_weight, grads->post_bias, grads->pre_weight, grads->pre_bias};
  int n_out = 0;
  for (int k = 0; k < kNumGrads; ++k)
    if (outs[k]) {
      a.want |= 1u << k;
      sum.out[n_out++] = outs[k];
    }
  a.chunks = grad_chunks(*c);
  a.gates = std::max(1, c->gates);
  const size_t need = (size_t)n_out * a.gates * a.chunks * c->channels * sizeof(float);
  if (need && (!workspace || workspace_bytes < need)) return HTTM_ERR_WORKSPACE;
  if (need && !aligned(workspace, 256)) return HTTM_ERR_ALIGN;
  a.partial = static_cast<float*>(workspace);
  a.gate = w->gate;
  a.post_w = w->post_weight, a.post_b = w->post_bias, a.pre_w = w->pre_weight, a.pre_b = w->pre_bias;
  a.stats = const_cast<float*>(stats);
  a.rows = c->rows;
  a.gate_rows = c->rows / a.gates;
  a.C = c->channels;
  a.post = c->post, a.pre = c->pre;
  a.rs = c->residual_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c->rows == 0 && !n_out) return HTTM_OK;
  HTTM_OPS_LAUNCH(by_type(*c, wide, [&](auto tx, auto tf, auto width) {
    return post ? launch_grad<decltype(tx), decltype(tf), decltype(width)::value, true>(a, s)
                : launch_grad<decltype(tx), decltype(tf), decltype(width)::value, false>(a, s);
  }), s);
  if (n_out) {
    sum.partial = a.partial;
    sum.is_gate0 = grads->gate != nullptr;
    sum.C = c->channels;
    sum.gates = a.gates;
    sum.chunks = a.chunks;
    const dim3 grid((c->channels + 15) / 16, n_out + (sum.is_gate0 ? a.gates - 1 : 0));
    norm_sum_kernel<<<grid, dim3(16, 64), 0, s>>>(sum);
    HTTM_OPS_LAUNCH(cudaGetLastError(), s);
  }
  return HTTM_OK;
}

}  // extern "C"
