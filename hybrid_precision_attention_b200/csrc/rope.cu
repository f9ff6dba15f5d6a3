// rope.cu — rotary positions of queries and keys in one launch.
//
// (u, v) -> amp * (u cos a - v sin a, v cos a + u sin a) on each pair of the
// first `rot` elements of a head, a = w_i * position.  The angle is kept as a
// fraction of a turn in 64-bit fixed point: position * freqs[i] modulo 2^64 is
// exact modulo one turn for every int32 position, where float32 angles are off
// by whole radians at the far end of long contexts and float64 ones cost 1/64
// of the float32 rate.  Its top 32 bits are signed half-turns, of which 24 go to
// sincospif: for 16-bit rows rounded, an error of at most pi * 2^-25 in the angle.  For
// float32 rows the other 8 turn its results on by a first-order step (their angle is below
// 2^-22), so that the angle's error is what is cut off, pi * 2^-31, and sines near 0 are
// right to their own last bits.
//
// Bound by memory: every element is read and written once.  A thread owns V
// pairs of one token (two V-element accesses, 16 bytes each on the vector path,
// from either half of the rotated elements, so that a warp's accesses run on in
// both layouts).  Many tokens: a block takes a few tokens with all their heads, its
// threads make the tokens' sines once, into shared memory, and each rotates its
// pairs of up to 8 heads, the first ones' loads in flight while the sines are made.
// Few tokens: a head a thread, the shortest chain (16 tokens 2.1 us, most of it the launch).
// 8192 tokens x 40 heads x 128, bf16: 31 us, 5.4 TB/s (a row pointer worked out for
// every head and each element converted by itself: 55 us); 5331 x 24 heads, f32: 22 us, 5.9 TB/s.
// Rows that 16-byte accesses do not divide take 2-element or single ones: rot 34 of 128, bf16, 4096
// x 40 heads 33 us, 2.5 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kv8.cuh"

namespace hq {
namespace {

struct RopeArgs {
  hq_rope_tensor t[2];
  int H0, H;           // heads of the first tensor, of both
  int T, D, rot, PG, CG;  // PG groups of V pairs, CG groups of 2V copied elements
  long long tokens;
  const int32_t* pos;
  const uint64_t* freqs;
  float amp, sign;
  int inplace[2];
  int TB, lanes;       // many tokens: tokens of a block, threads that share a group's heads
};

template <class E, int V>
struct alignas(sizeof(E) * V) Vec {
  E e[V];
};

// Where group g of a head has its two V-element accesses.  Copied elements: the
// second access may lie past D.  Single elements of an interleaved pair (V = 1)
// stand side by side.
template <int V, bool HALF>
struct Place {
  int d0, d1;
  bool turn, two;
  __device__ __forceinline__ Place(const RopeArgs& a, int g) {
    constexpr bool SIDE = !HALF && V == 1;
    turn = g < a.PG;
    d0 = turn ? (SIDE ? 2 * g : g * V) : a.rot + (g - a.PG) * V;
    d1 = turn ? (SIDE ? d0 + 1 : a.rot / 2 + g * V) : d0 + a.CG * V;
    two = d1 < a.D;
  }
  // pair i of the group.  half, or single elements: g V + i; interleaved: V / 2 pairs of each access
  __device__ __forceinline__ int pair(int i) const { return HALF || V == 1 ? (V == 1 && !HALF ? d0 / 2 : d0 + i) : (i < V / 2 ? d0 / 2 + i : d1 / 2 + i - V / 2); }
};

template <class E>
__device__ __forceinline__ float2 sine(const RopeArgs& a, long long tok, int pair) {  // (cos, sin) with their factors
  const uint64_t turns = static_cast<uint64_t>(static_cast<long long>(a.pos[tok])) * a.freqs[pair];
  const uint32_t t = static_cast<uint32_t>(turns >> 32);
  // float32: to a multiple of 256 (past the last one a whole turn on)
  const uint32_t top = sizeof(E) == 4 ? (t + 128u) & ~255u : t;
  float c, s;
  sincospif(static_cast<float>(static_cast<int32_t>(top)) * 0x1p-31f, &s, &c);
  if (sizeof(E) == 4) {
    const float rest = static_cast<float>(static_cast<int32_t>(t - top)) * 1.46291808e-9f /* pi 2^-31 */, c0 = c;
    c = fmaf(-s, rest, c);
    s = fmaf(c0, rest, s);
  }
  return make_float2(c * a.amp, s * a.sign);
}

// two 16-bit elements in a word
template <class E>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (IsBf16<E>::value) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <class E>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  uint32_t w;
  if (IsBf16<E>::value) *reinterpret_cast<__nv_bfloat162*>(&w) = __floats2bfloat162_rn(x, y);
  else *reinterpret_cast<__half2*>(&w) = __floats2half2_rn(x, y);
  return w;
}

template <class E, int V, bool HALF>
__device__ __forceinline__ void rotate(Vec<E, V>& u, Vec<E, V>& w, const float2 (&cs)[V]) {
  if constexpr (sizeof(E) == 2 && V % 2 == 0) {
    uint32_t* a = reinterpret_cast<uint32_t*>(u.e);
    uint32_t* b = reinterpret_cast<uint32_t*>(w.e);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 x = unpack2<E>(a[i]), y = unpack2<E>(b[i]);
      if (HALF) {  // pairs (x.x, y.x), (x.y, y.y)
        const float2 p = cs[2 * i], q = cs[2 * i + 1];
        a[i] = pack2<E>(x.x * p.x - y.x * p.y, x.y * q.x - y.y * q.y);
        b[i] = pack2<E>(y.x * p.x + x.x * p.y, y.y * q.x + x.y * q.y);
      } else {     // pairs (x.x, x.y), (y.x, y.y)
        const float2 p = cs[i], q = cs[V / 2 + i];
        a[i] = pack2<E>(x.x * p.x - x.y * p.y, x.y * p.x + x.x * p.y);
        b[i] = pack2<E>(y.x * q.x - y.y * q.y, y.y * q.x + y.x * q.y);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // half: pair i = (u[i], w[i]); interleaved: elements 2i, 2i+1 of u, then of w
      E& eu = HALF || V == 1 ? u.e[i] : (2 * i < V ? u.e[(2 * i) % V] : w.e[(2 * i) % V]);
      E& ev = HALF || V == 1 ? w.e[i] : (2 * i + 1 < V ? u.e[(2 * i + 1) % V] : w.e[(2 * i + 1) % V]);
      const float fu = to_float(eu), fv = to_float(ev);
      eu = from_float<E>(fu * cs[i].x - fv * cs[i].y);
      ev = from_float<E>(fv * cs[i].x + fu * cs[i].y);
    }
  }
}

// the head's row in x (`in`) or y
template <class E>
__device__ __forceinline__ E* row_of(const RopeArgs& a, int h, long long b, long long t, bool in) {
  const int z = h >= a.H0;
  const hq_rope_tensor& x = a.t[z];
  return in ? const_cast<E*>(static_cast<const E*>(x.x)) + b * x.x_batch + t * x.x_tok + (h - z * a.H0) * x.x_head
            : static_cast<E*>(x.y) + b * x.y_batch + t * x.y_tok + (h - z * a.H0) * x.y_head;
}

template <class E, int V, bool HALF>
__global__ void __launch_bounds__(256) rope_few_kernel(const __grid_constant__ RopeArgs a) {
  chained();
  const int per = a.PG + a.CG, g = threadIdx.x % per;
  const long long tok = static_cast<long long>(blockIdx.x) * (blockDim.x / per) + threadIdx.x / per;
  const int h = blockIdx.y, z = h >= a.H0;
  if (threadIdx.x >= blockDim.x / per * per || tok >= a.tokens) return;
  const Place<V, HALF> at(a, g);
  if (!at.turn && a.inplace[z]) return;
  const long long b = tok / a.T, t = tok - b * a.T;
  const E* p = row_of<E>(a, h, b, t, true);
  Vec<E, V> u = *reinterpret_cast<const Vec<E, V>*>(p + at.d0), w = {};
  if (at.two) w = *reinterpret_cast<const Vec<E, V>*>(p + at.d1);
  if (at.turn) {
    float2 cs[V];
#pragma unroll
    for (int i = 0; i < V; ++i) cs[i] = sine<E>(a, tok, at.pair(i));
    rotate<E, V, HALF>(u, w, cs);
  }
  E* q = row_of<E>(a, h, b, t, false);
  *reinterpret_cast<Vec<E, V>*>(q + at.d0) = u;
  if (at.two) *reinterpret_cast<Vec<E, V>*>(q + at.d1) = w;
}

constexpr int HPT = 2;       // heads of a thread at a time (4: fewer threads fit, 35 us against 31 us)
constexpr int HEADS = 8;     // heads of a thread, where there are threads enough

template <class E, int V, bool HALF>
__global__ void __launch_bounds__(256) rope_many_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 table[256 * V];   // (cos, sin) of [token of the block][pair]
  chained();
  const int per = a.PG + a.CG, slots = 256 / per, pairs = a.rot / 2;
  const int g = threadIdx.x % per, slot = threadIdx.x / per;
  const int k = slot / a.lanes, lane = slot - k * a.lanes;  // token of the block; the thread's heads: lane, lane + lanes, ..
  const long long tok0 = static_cast<long long>(blockIdx.x) * a.TB, tok = tok0 + k;
  const bool mine = slot < slots && k < a.TB && tok < a.tokens;
  const Place<V, HALF> at(a, g);
  const long long b = mine ? tok / a.T : 0, t = mine ? tok - b * a.T : 0;
  // the thread's heads of tensor z, HPT at a time; row pointers step from head to
  // head of the thread (a multiplication per head and tensor cost as much as the rotation)
  Vec<E, V> u[HPT], w[HPT];
  auto load = [&](const E* p, int64_t step, int n, bool any) {
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
      if (j < n && any) {
        u[j] = *reinterpret_cast<const Vec<E, V>*>(p + j * step + at.d0);
        if (at.two) w[j] = *reinterpret_cast<const Vec<E, V>*>(p + j * step + at.d1);
      }
    }
  };
  auto heads = [&](int H) { return mine && lane < H ? (H - lane + a.lanes - 1) / a.lanes : 0; };
  auto in_row = [&](const hq_rope_tensor& x) { return static_cast<const E*>(x.x) + b * x.x_batch + t * x.x_tok + lane * x.x_head; };
  load(in_row(a.t[0]), a.lanes * a.t[0].x_head, heads(a.H0), at.turn || !a.inplace[0]);
  const int here = static_cast<int>(min(static_cast<long long>(a.TB), a.tokens - tok0));
  for (int i = threadIdx.x; i < here * pairs; i += 256) {
    const int q = i / pairs;
    table[i] = sine<E>(a, tok0 + q, i - q * pairs);
  }
  __syncthreads();
  if (!mine) return;
  float2 cs[V];
  if (at.turn) {
#pragma unroll
    for (int i = 0; i < V; ++i) cs[i] = table[k * pairs + at.pair(i)];
  }
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const hq_rope_tensor& x = a.t[z];
    int n = heads(z ? a.H - a.H0 : a.H0);
    if (n == 0 || (!at.turn && a.inplace[z])) continue;
    const int64_t si = a.lanes * x.x_head, so = a.lanes * x.y_head;
    const E* p = in_row(x);
    E* q = static_cast<E*>(x.y) + b * x.y_batch + t * x.y_tok + lane * x.y_head;
    for (bool first = z == 0; n > 0; n -= HPT, p += HPT * si, q += HPT * so, first = false) {
      if (!first) load(p, si, n, true);
#pragma unroll
      for (int j = 0; j < HPT; ++j) {
        if (j >= n) break;
        if (at.turn) rotate<E, V, HALF>(u[j], w[j], cs);
        *reinterpret_cast<Vec<E, V>*>(q + j * so + at.d0) = u[j];
        if (at.two) *reinterpret_cast<Vec<E, V>*>(q + j * so + at.d1) = w[j];
      }
    }
  }
}

template <class E, int V, bool HALF>
hq_status launch_v(RopeArgs& a, cudaStream_t st) {
  a.PG = a.rot / 2 / V;
  const bool copy = !a.inplace[0] || (a.H > a.H0 && !a.inplace[1]);
  a.CG = copy ? ((a.D - a.rot) / V + 1) / 2 : 0;
  const int per = a.PG + a.CG;
  // a block holds whole tokens (per <= 256: D <= HQ_ROPE_MAX_DIM)
  const int slots = 256 / per;
  const int lanes = std::min((a.H + HEADS - 1) / HEADS, slots);
  a.TB = slots / lanes;
  a.lanes = lanes;
  const long long many = (a.tokens + a.TB - 1) / a.TB, few = (a.tokens + slots - 1) / slots;
  if (few > 0x7fffffffll || many > 0x7fffffffll) return HQ_ERR_UNSUPPORTED;
  // heads share their sines from half as many blocks as SMs on (40 heads x 128, bf16: 592
  // tokens 4.8 us against 5.3 us, 1184 6.0 against 8.0; 300 tokens 4.8 against 4.4, 16 4.6 against 2.0)
  if (many >= 148 / 2) {
    return cuda_status(launch_chained(rope_many_kernel<E, V, HALF>, dim3(static_cast<unsigned>(many)), 256, 0, st, a), "rope launch");
  } else {
    if (a.H > 65535) return HQ_ERR_UNSUPPORTED;
    return cuda_status(launch_chained(rope_few_kernel<E, V, HALF>, dim3(static_cast<unsigned>(few), a.H), 256, 0, st, a), "rope launch");
  }
}

template <class E, bool HALF>
hq_status launch_e(RopeArgs& a, cudaStream_t st) {
  // the widest access that every row of x and y, the pairs and the rest divide into
  auto fits = [&](int V) {
    if (a.rot / 2 % V || a.D % V) return false;
    for (int z = 0; z < (a.H > a.H0 ? 2 : 1); ++z) {
      const hq_rope_tensor& x = a.t[z];
      const int64_t all = x.x_batch | x.x_tok | x.x_head | x.y_batch | x.y_tok | x.y_head;
      if (all % V || (reinterpret_cast<uintptr_t>(x.x) | reinterpret_cast<uintptr_t>(x.y)) % (V * sizeof(E))) return false;
    }
    return true;
  };
  constexpr int W = 16 / sizeof(E);
  if (fits(W)) return launch_v<E, W, HALF>(a, st);
  if (fits(2)) return launch_v<E, 2, HALF>(a, st);
  return launch_v<E, 1, HALF>(a, st);
}

template <class E>
hq_status launch_l(RopeArgs& a, int layout, cudaStream_t st) {
  return layout == HQ_ROPE_HALF ? launch_e<E, true>(a, st) : launch_e<E, false>(a, st);
}

}  // namespace
}  // namespace hq

extern "C" {

hq_status hq_rope_freqs(int32_t rot, double base, int32_t kind, double factor, double orig_len, double low, double high,
                        uint64_t* freqs, float* amp) {
  if (!freqs || !amp || rot < 2 || rot % 2 || rot > 65536 || !(base > 1.0) || !std::isfinite(base)) return HQ_ERR_INVALID;
  if (kind < HQ_ROPE_PLAIN || kind > HQ_ROPE_BANDS) return HQ_ERR_INVALID;
  if (kind != HQ_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return HQ_ERR_INVALID;
  if (kind == HQ_ROPE_NTK && rot == 2) return HQ_ERR_INVALID;
  if (kind == HQ_ROPE_YARN || kind == HQ_ROPE_BANDS) {
    if (low == 0) low = 1;
    if (high == 0) high = kind == HQ_ROPE_YARN ? 32 : 4;
    if (!(orig_len > 0) || !std::isfinite(orig_len) || !(low > 0) || !(high > low) || !std::isfinite(high)) return HQ_ERR_INVALID;
  }
  // long double: 11 more bits than the fixed-point fraction keeps of a float64
  typedef long double L;
  const L two_pi = 6.283185307179586476925286766559005768L;
  L bs = base, a = 0, c = 1;
  if (kind == HQ_ROPE_NTK) bs *= powl(factor, static_cast<L>(rot) / (rot - 2));
  if (kind == HQ_ROPE_YARN) {
    const L per = rot / (2 * logl(bs));
    a = fmaxl(floorl(per * logl(orig_len / (two_pi * high))), 0);
    c = fminl(ceill(per * logl(orig_len / (two_pi * low))), rot - 1);
  }
  *amp = kind == HQ_ROPE_YARN && factor > 1 ? static_cast<float>(1.0 + 0.1 * std::log(factor)) : 1.0f;
  for (int i = 0; i < rot / 2; ++i) {
    L w = powl(bs, static_cast<L>(-2 * i) / rot);
    if (kind == HQ_ROPE_LINEAR) w /= factor;
    if (kind == HQ_ROPE_YARN) {
      const L r = fminl(fmaxl((i - a) / fmaxl(c - a, 0.001L), 0), 1);
      w = w / factor * r + w * (1 - r);
    }
    if (kind == HQ_ROPE_BANDS) {
      const L r = fminl(fmaxl((orig_len * w / two_pi - low) / (static_cast<L>(high) - low), 0), 1);
      w = (1 - r) * w / factor + r * w;
    }
    freqs[i] = static_cast<uint64_t>(ldexpl(w / two_pi, 64) + 0.5L);  // w <= 1: below 2^62
  }
  return HQ_OK;
}

hq_status hq_rope(int32_t dtype, int32_t B, int32_t T, int32_t D, int32_t rot, int32_t layout, int32_t grad,
                  const hq_rope_tensor* q, const hq_rope_tensor* k, const int32_t* pos, const uint64_t* freqs, float amp,
                  hq_stream_t stream) {
  if (dtype < HQ_F16 || dtype > HQ_F32 || (layout != HQ_ROPE_HALF && layout != HQ_ROPE_INTERLEAVED)) return HQ_ERR_INVALID;
  if (!q || B < 0 || T < 0 || D < 1 || rot < 2 || rot % 2 || rot > D) return HQ_ERR_INVALID;
  if (D > HQ_ROPE_MAX_DIM) return HQ_ERR_UNSUPPORTED;
  const size_t es = dtype == HQ_F32 ? 4 : 2;
  hq::RopeArgs a = {};
  const hq_rope_tensor* both[2] = {q, k};
  for (int z = 0; z < 2; ++z) {
    const hq_rope_tensor* x = both[z];
    if (!x) continue;
    if (x->H < 0) return HQ_ERR_INVALID;
    if (x->H > 0 && B > 0 && T > 0 &&
        (!x->x || !x->y || (reinterpret_cast<uintptr_t>(x->x) | reinterpret_cast<uintptr_t>(x->y)) % es))
      return HQ_ERR_INVALID;
    hq_rope_tensor& y = a.t[z];
    y = *x;
    // the stride of a dimension of one is never used, whatever it says
    if (B <= 1) y.x_batch = y.y_batch = 0;
    if (T <= 1) y.x_tok = y.y_tok = 0;
    if (y.H <= 1) y.x_head = y.y_head = 0;
    a.inplace[z] = y.x == y.y;
    // in place, every element must be read where it is written
    if (a.inplace[z] && B > 0 && T > 0 && x->H > 0 && (y.x_batch != y.y_batch || y.x_tok != y.y_tok || y.x_head != y.y_head)) return HQ_ERR_INVALID;
  }
  a.H0 = q->H;
  a.H = q->H + (k ? k->H : 0);
  if (B == 0 || T == 0 || a.H == 0) return HQ_OK;
  if (!pos || (reinterpret_cast<uintptr_t>(pos) & 3u) || !freqs || (reinterpret_cast<uintptr_t>(freqs) & 7u)) return HQ_ERR_INVALID;
  a.T = T;
  a.D = D;
  a.rot = rot;
  a.tokens = static_cast<long long>(B) * T;
  a.pos = pos;
  a.freqs = freqs;
  a.amp = amp;
  a.sign = grad ? -amp : amp;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == HQ_F16) return hq::launch_l<__half>(a, layout, st);
  if (dtype == HQ_BF16) return hq::launch_l<__nv_bfloat16>(a, layout, st);
  return hq::launch_l<float>(a, layout, st);
}

}  // extern "C"
