// Rotary positions: pairs of channels turned by position * frequency, from
// any strided layout into any other (a packed projection into [h, N, d]).
//
// The operator is bound by memory: every element is read and written once.
// An angle belongs to (token, pair) and serves every head, so a thread owns
// W pairs of one token, computes their cosines and sines once, and walks
// over the heads of both tensors.  Four neighbouring threads of a 64-channel
// head read and write whole 128-byte rows.  When there are few tokens the
// heads are divided among more threads.
//
// Angles: frequencies are given in radians per position (fp64).  In turns
// and 64-bit fixed point, position * frequency is one integer product whose
// overflow drops whole turns exactly, and so do its top bits the quarters.
// What is left is the fp64 rounding of the frequency in turns (2^-52 of it,
// times the position) and the fp32 rounding of the rest, an eighth of a turn
// at most: 2^-28 turns.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "ops.h"

namespace httm {
namespace {

struct RotaryArgs {
  View in[2], out[2];           // queries, keys
  int heads[2];
  int batch, tokens, axes, pairs, d, rot;
  int chunks, tail_chunks;      // W-pair chunks of a head, W-channel chunks of what is copied
  int head_groups, heads_per;   // the heads divided among threads
  const int32_t* pos;
  int64_t pos_batch;
  const double* freqs;
  float factor;
  int inverse;
};

// W consecutive elements as they lie in memory; W = 8 goes in 16-byte accesses.
template <class T, int W>
struct Vec {
  static constexpr int n = W == 1 ? 1 : W * (int)sizeof(T) / 4;
  uint32_t w[n];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (W == 1) {
      w[0] = __float_as_uint(to_f(*p));
    } else {
#pragma unroll
      for (int i = 0; i < n / 4; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[W]) const {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      if constexpr (W == 1 || sizeof(T) == 4) v[e] = __uint_as_float(w[e]);
      else v[e] = __uint_as_float((e & 1) ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
  }
};
template <class T, int W>
__device__ __forceinline__ void store_w(T* p, const float (&v)[W]) {
  if constexpr (W == 1) {
    *p = from_f<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// cos and sin of pos * freq (freq in radians per position, any sign).
__device__ __forceinline__ void turn(double freq, int pos, float factor, bool inverse, float& c, float& s) {
  // turns per position as a 64-bit fraction of one turn (whole turns drop out)
  const double t = freq * 0.15915494309189533577;            // 1 / (2 pi)
  const double frac = t - floor(t);
  const unsigned long long step = __double2ull_rn(frac * 18446744073709551616.0);   // 1.0 saturates to 2^64 - 1
  const unsigned long long phase = step * (unsigned long long)(long long)pos;
  // the nearest quarter turn, and the rest in half turns: [-1/4, 1/4]
  const unsigned quarter = (unsigned)((phase + (1ull << 61)) >> 62);
  const int high = (int)((uint32_t)(phase >> 32) - (quarter << 30));
  const float rest = fmaf((float)high, 0x1p-31f, (float)(uint32_t)phase * 0x1p-63f);
  float cr, sr;
  sincospif(rest, &sr, &cr);
  c = quarter & 1 ? sr : cr;
  s = quarter & 1 ? cr : sr;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter >= 2) s = -s;
  c *= factor;
  s *= inverse ? -factor : factor;
}

// (a, b) turned: the products are contracted by hand, so that every path
// gives the same bits.
__device__ __forceinline__ void turn_pair(float a, float b, float c, float s, float& x, float& y) {
  x = fmaf(a, c, -__fmul_rn(b, s));
  y = fmaf(b, c, __fmul_rn(a, s));
}

// heads read ahead: 185 us without, 139 with 4, 130 with 8 (41,070 tokens x 32
// heads, twice, in one group); the element accesses of odd shapes are slower with 8
template <int W>
constexpr int kHeadsAhead = W == 8 ? 8 : 4;

template <class T, int W, bool HALF>
__global__ void __launch_bounds__(256) rotary_kernel(RotaryArgs a) {
  const int per_token = a.chunks + a.tail_chunks;
  const long long total = (long long)a.batch * a.head_groups * a.tokens * per_token;
  const long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (at >= total) return;
  int ch, tok, hg, b;
  if (total <= 0x7fffffffll) {             // 32-bit divisions where they do
    uint32_t i = (uint32_t)at;
    ch = i % (uint32_t)per_token, i /= (uint32_t)per_token;
    tok = i % (uint32_t)a.tokens, i /= (uint32_t)a.tokens;
    hg = i % (uint32_t)a.head_groups, b = i / (uint32_t)a.head_groups;
  } else {
    long long i = at;
    ch = (int)(i % per_token), i /= per_token;
    tok = (int)(i % a.tokens), i /= a.tokens;
    hg = (int)(i % a.head_groups), b = (int)(i / a.head_groups);
  }
  const bool copied = ch >= a.chunks;

  float c[W], s[W];
  int lo, hi;                              // first channel of the two runs of W this thread handles
  if (copied) {
    lo = a.rot + (ch - a.chunks) * W;
    hi = lo;
  } else {
    const int p0 = ch * W;                 // first pair, counted over all axes
    if (HALF) {                            // W divides the pairs of an axis: one axis per chunk
      const int ax = p0 / a.pairs, n = p0 - ax * a.pairs;
      lo = ax * 2 * a.pairs + n;
      hi = lo + a.pairs;
    } else {
      lo = 2 * p0;
      hi = lo + W;
    }
    const int32_t* pos = a.pos + b * a.pos_batch + (long long)tok * a.axes;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int ax = (p0 + e) / a.pairs, n = p0 + e - ax * a.pairs;
      turn(a.freqs[n], pos[ax], a.factor, a.inverse != 0, c[e], s[e]);
    }
  }

  // several heads are read before the first of them is written (in place, a
  // thread writes only what it has read)
  const int h0 = hg * a.heads_per, h1 = min(h0 + a.heads_per, a.heads[0] + a.heads[1]);
  auto row = [&](const View (&v)[2], int h) {
    const int which = h >= a.heads[0] ? 1 : 0;
    return reinterpret_cast<T*>(v[which].data) + b * v[which].sb + (h - (which ? a.heads[0] : 0)) * v[which].sh +
           tok * v[which].st;
  };
  constexpr int kBatch = kHeadsAhead<W>;
  for (int h = h0; h < h1; h += kBatch) {
    Vec<T, W> x[kBatch], y[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (h + i < h1) {
        const T* src = row(a.in, h + i);
        x[i].load(src + lo);
        if (!copied) y[i].load(src + hi);
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (h + i < h1) {
        T* dst = row(a.out, h + i);
        float u[W], v[W];
        x[i].get(u);
        if (copied) {
          store_w<T, W>(dst + lo, u);
          continue;
        }
        y[i].get(v);
        float p[W], q[W];
        if constexpr (HALF || W == 1) {
#pragma unroll
          for (int e = 0; e < W; ++e) turn_pair(u[e], v[e], c[e], s[e], p[e], q[e]);
        } else {                           // pairs lie side by side in the 2 W channels (u, v)
#pragma unroll
          for (int e = 0; e < W / 2; ++e) {
            turn_pair(u[2 * e], u[2 * e + 1], c[e], s[e], p[2 * e], p[2 * e + 1]);
            turn_pair(v[2 * e], v[2 * e + 1], c[e + W / 2], s[e + W / 2], q[2 * e], q[2 * e + 1]);
          }
        }
        store_w<T, W>(dst + lo, p);
        store_w<T, W>(dst + hi, q);
      }
  }
}

template <class T, int W>
cudaError_t launch_w(RotaryArgs& a, bool half, cudaStream_t s) {
  a.chunks = a.axes * a.pairs / W;
  a.tail_chunks = (a.d - a.rot) / W;
  const long long work = (long long)a.batch * a.tokens * (a.chunks + a.tail_chunks);
  const int heads = a.heads[0] + a.heads[1];
  // a thread per (token, chunk) walks over all heads once there are enough
  // of them for the loads in flight that the memory needs (about 1,024
  // threads an SM); with fewer tokens the heads are divided
  const long long want = (long long)kSMs * 1024;
  a.head_groups = (int)std::min<long long>(heads, std::max<long long>(1, (want + work - 1) / work));
  if (W == 8 && a.head_groups == 1) {
    // ... or as far as it fills the last wave of 512 threads an SM: a thread
    // costs its batches of heads and 0.45 of one for its angles (41,070 tokens
    // x 32 heads, twice, in 1 / 2 / 3 / 4 groups: 130 / 122 / 131 / 130 us)
    double best = 0;
    for (int g = 1; g <= std::min(heads, 4); ++g) {
      const long long waves = (work * g + kSMs * 512 - 1) / (kSMs * 512);
      const int per = (heads + g - 1) / g;
      const double cost = (double)waves * ((per + kHeadsAhead<W> - 1) / kHeadsAhead<W> + 0.45);
      if (g == 1 || cost < best) best = cost, a.head_groups = g;
    }
  }
  a.heads_per = (heads + a.head_groups - 1) / a.head_groups;
  a.head_groups = (heads + a.heads_per - 1) / a.heads_per;
  const int threads = work * a.head_groups < kSMs * 256 ? 64 : 256;
  const long long grid = (work * a.head_groups + threads - 1) / threads;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (half)
    rotary_kernel<T, W, true><<<(unsigned)grid, threads, 0, s>>>(a);
  else
    rotary_kernel<T, W, false><<<(unsigned)grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_t(RotaryArgs& a, bool half, cudaStream_t s) {
  // 8 channels at a time where every run is a multiple of 8 and every row
  // starts on 16 bytes; else one pair at a time
  const int el = 16 / (int)sizeof(T);
  bool wide = a.d % 8 == 0 && a.rot % 16 == 0 && (half ? a.pairs % 8 == 0 : true);
  for (int w = 0; w < (a.heads[1] ? 2 : 1); ++w)
    for (const View* v : {&a.in[w], &a.out[w]})
      wide = wide && aligned(v->data, 16) && v->sb % el == 0 && v->sh % el == 0 && v->st % el == 0;
  return wide ? launch_w<T, 8>(a, half, s) : launch_w<T, 1>(a, half, s);
}

}  // namespace
}  // namespace httm

using namespace httm;

extern "C" httm_status httm_rotary(const httm_rotary_cfg* c, const httm_view* q, const httm_view* q_out,
                                   const httm_view* k, const httm_view* k_out, void* stream) {
  if (!c || !q || !q_out) return HTTM_ERR_ARG;
  if (c->batch < 0 || c->tokens < 0 || c->heads < 1 || c->kv_heads < 0) return HTTM_ERR_ARG;
  if (c->d_head < 1 || c->axes < 1 || c->axes > 4 || c->pairs < 1) return HTTM_ERR_ARG;
  if (2ll * c->axes * c->pairs > c->d_head) return HTTM_ERR_ARG;
  if (c->layout != HTTM_ROTARY_HALF && c->layout != HTTM_ROTARY_PAIRS) return HTTM_ERR_ARG;
  if (c->dtype != HTTM_BF16 && c->dtype != HTTM_F32) return HTTM_ERR_ARG;
  if (c->position_batch < 0 || !(c->factor - c->factor == 0.f)) return HTTM_ERR_ARG;
  if (c->d_head > 1024) return HTTM_ERR_UNSUPPORTED;
  if ((long long)c->heads + c->kv_heads > (1 << 20)) return HTTM_ERR_UNSUPPORTED;
  if (c->kv_heads > 0 && (!k || !k_out)) return HTTM_ERR_ARG;
  if (c->batch == 0 || c->tokens == 0) return HTTM_OK;
  if (!c->positions || !c->freqs) return HTTM_ERR_ARG;
  if (!aligned(c->positions, 4) || !aligned(c->freqs, 8)) return HTTM_ERR_ALIGN;
  const size_t es = c->dtype == HTTM_F32 ? 4 : 2;
  RotaryArgs a{};
  const int heads[2] = {c->heads, c->kv_heads};
  const httm_view* in[2] = {q, k};
  const httm_view* out[2] = {q_out, k_out};
  for (int w = 0; w < 2; ++w) {
    a.heads[w] = heads[w];
    if (heads[w] == 0) continue;
    for (const httm_view* v : {in[w], out[w]}) {
      if (!v->data || v->batch < 0 || v->head < 0 || v->token < 0) return HTTM_ERR_ARG;
      if (!aligned(v->data, es)) return HTTM_ERR_ALIGN;
    }
    a.in[w] = normal_view(*in[w], c->batch, heads[w], c->tokens);
    a.out[w] = normal_view(*out[w], c->batch, heads[w], c->tokens);
    if (!disjoint(a.out[w], c->batch, heads[w], c->tokens, c->d_head)) return HTTM_ERR_ARG;
  }
  a.batch = c->batch;
  a.tokens = c->tokens;
  a.axes = c->axes;
  a.pairs = c->pairs;
  a.d = c->d_head;
  a.rot = 2 * c->axes * c->pairs;
  a.pos = c->positions;
  a.pos_batch = c->position_batch;
  a.freqs = c->freqs;
  a.factor = c->factor;
  a.inverse = c->inverse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = c->layout == HTTM_ROTARY_HALF;
  HTTM_OPS_LAUNCH(c->dtype == HTTM_F32 ? launch_t<float>(a, half, s) : launch_t<__nv_bfloat16>(a, half, s), s);
  return HTTM_OK;
}
