// rope.cu — rotary positions of queries and keys in one launch.
//
// (u, v) -> amp * (u cos a - v sin a, v cos a + u sin a) on each pair of the
// first `rot` elements of a head, a = w_i * position.  The angle is kept as a
// fraction of a turn in 64-bit fixed point: position * freqs[i] modulo 2^64 is
// exact modulo one turn for every int32 position, where float32 angles are off
// by whole radians at the far end of long contexts and float64 ones cost 1/64
// of the float32 rate.  Its top 32 bits, taken as signed half-turns, go to
// sincospif: the angle's own error is at most pi * 2^-25.
//
// Bound by memory: every element is read and written once.  A thread owns V
// pairs (two V-element accesses, 16 bytes each on the vector path) of one token
// and rotates them for HPT heads, so that the V sincospif of a token's pairs
// are shared by those heads and all of the thread's loads are in flight while
// they are computed.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

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
};

template <class E, int V>
struct alignas(sizeof(E) * V) Vec {
  E e[V];
};

template <class E, int V, int HPT, bool HALF>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
  const int per = a.PG + a.CG;
  const int g = threadIdx.x % per;
  const long long tok = static_cast<long long>(blockIdx.x) * (blockDim.x / per) + threadIdx.x / per;
  if (threadIdx.x >= blockDim.x / per * per || tok >= a.tokens) return;
  const long long b = tok / a.T, t = tok - b * a.T;
  const bool turn = g < a.PG;
  // the group's two V-element accesses within a head; copied elements: the
  // second access may lie past D
  const int d0 = turn ? (HALF ? g * V : 2 * g * V) : a.rot + 2 * (g - a.PG) * V;
  const int d1 = turn && HALF ? a.rot / 2 + g * V : d0 + V;
  const bool two = d1 < a.D;

  Vec<E, V> u[HPT], w[HPT];
  const int h0 = blockIdx.y * HPT;
#pragma unroll
  for (int k = 0; k < HPT; ++k) {
    const int h = h0 + k;
    if (h < a.H) {
      const int z = h >= a.H0;
      const hq_rope_tensor& x = a.t[z];
      if (turn || !a.inplace[z]) {
        const E* p = static_cast<const E*>(x.x) + b * x.x_batch + t * x.x_tok + (h - z * a.H0) * x.x_head;
        u[k] = *reinterpret_cast<const Vec<E, V>*>(p + d0);
        if (two) w[k] = *reinterpret_cast<const Vec<E, V>*>(p + d1);
      }
    }
  }
  float c[V], s[V];
  if (turn) {
    const long long pos = a.pos[tok];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t turns = static_cast<uint64_t>(pos) * a.freqs[g * V + i];
      sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f /* 2^-31 */, &s[i], &c[i]);
      c[i] *= a.amp;
      s[i] *= a.sign;
    }
  }
#pragma unroll
  for (int k = 0; k < HPT; ++k) {
    const int h = h0 + k;
    if (h >= a.H) break;
    const int z = h >= a.H0;
    const hq_rope_tensor& x = a.t[z];
    if (turn) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // half: pair i = (u[i], w[i]); interleaved: pair i = elements 2i, 2i+1 of (u, w) in a row
        E& eu = HALF ? u[k].e[i] : (2 * i < V ? u[k].e[(2 * i) % V] : w[k].e[(2 * i) % V]);
        E& ev = HALF ? w[k].e[i] : (2 * i + 1 < V ? u[k].e[(2 * i + 1) % V] : w[k].e[(2 * i + 1) % V]);
        const float fu = to_float(eu), fv = to_float(ev);
        eu = from_float<E>(fu * c[i] - fv * s[i]);
        ev = from_float<E>(fv * c[i] + fu * s[i]);
      }
    } else if (a.inplace[z]) {
      continue;
    }
    E* p = static_cast<E*>(x.y) + b * x.y_batch + t * x.y_tok + (h - z * a.H0) * x.y_head;
    *reinterpret_cast<Vec<E, V>*>(p + d0) = u[k];
    if (two) *reinterpret_cast<Vec<E, V>*>(p + d1) = w[k];
  }
}

template <class E, int V, bool HALF>
hq_status launch_v(RopeArgs& a, cudaStream_t st) {
  a.PG = a.rot / 2 / V;
  const bool copy = !a.inplace[0] || (a.H > a.H0 && !a.inplace[1]);
  a.CG = copy ? ((a.D - a.rot) / V + 1) / 2 : 0;
  const int per = a.PG + a.CG;
  // a block holds whole tokens (per <= 256: D <= HQ_ROPE_MAX_DIM)
  constexpr int threads = 256;
  const int tb = threads / per;
  const long long blocks = (a.tokens + tb - 1) / tb;
  if (blocks > 0x7fffffffll) return HQ_ERR_UNSUPPORTED;
  // Heads per thread: 4 share a thread's sines once that still leaves enough
  // warps to fill the GPU; few tokens take 1, the shortest chain per thread.
  const bool wide = blocks * ((a.H + 3) / 4) >= 2 * 148;
  const dim3 grid(static_cast<unsigned>(blocks), (a.H + (wide ? 4 : 1) - 1) / (wide ? 4 : 1));
  if (grid.y > 65535u) return HQ_ERR_UNSUPPORTED;
  if (wide)
    rope_kernel<E, V, 4, HALF><<<grid, threads, 0, st>>>(a);
  else
    rope_kernel<E, V, 1, HALF><<<grid, threads, 0, st>>>(a);
  return cuda_status(cudaGetLastError(), "rope launch");
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
    if (a.inplace[z] && (y.x_batch != y.y_batch || y.x_tok != y.y_tok || y.x_head != y.y_head)) return HQ_ERR_INVALID;
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
