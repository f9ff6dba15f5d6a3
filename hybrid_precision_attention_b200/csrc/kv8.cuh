// kv8.cuh — what the kernels of the 8-bit block cache share: element types,
// page addressing, and the quantisers of a block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace hq {

constexpr int KV8_BLOCK = 64;                      // positions of a page

// ----------------------------------------------------------------- pairs of floats in one register pair

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f32x2_split(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }
template <class E>
__device__ __forceinline__ E from_float(float x);
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }

template <class E>
struct IsBf16 {
  static constexpr bool value = false;
};
template <>
struct IsBf16<__nv_bfloat16> {
  static constexpr bool value = true;
};

// Launch with programmatic dependent launch: the grid may start while the one before
// it in the stream drains.  Every CTA of such a kernel calls chained() before it
// touches memory: it waits until the grids before have completed, then lets the next
// one start in turn.  (Kernels of 2 to 20 us, one behind another: 1 to 2 us less each.)
template <class K, class A>
inline cudaError_t launch_chained(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, const A& arg) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, arg);
}
__device__ __forceinline__ void chained() {
  griddep_wait();
  griddep_launch_dependents();
}

// Pool index of page j of (b, kv head) bh, -1 when the table's entry lies outside the pool.
__device__ __forceinline__ long long kv8_page_index(const hq_kv8_cache& c, size_t bh, int j) {
  const size_t npg = static_cast<size_t>(c.cap / KV8_BLOCK);
  if (c.page_table == nullptr) return static_cast<long long>(bh * npg + j);
  const int idx = c.page_table[bh * npg + j];
  return (idx >= 0 && idx < c.n_pages) ? idx : -1;
}
__device__ __forceinline__ void kv8_err(const hq_kv8_cache& c, int b, uint32_t bit) {
  atomicOr(reinterpret_cast<unsigned int*>(c.err + b), bit);
}
// For readers: an entry outside the pool is flagged and pool page 0 is read instead.
__device__ __forceinline__ const uint8_t* kv8_page(const hq_kv8_cache& c, size_t bh, int j) {
  const long long idx = kv8_page_index(c, bh, j);
  if (idx < 0) {
    kv8_err(c, static_cast<int>(bh / c.Hkv), HQ_DEVERR_PAGE);
    return c.pages;
  }
  return c.pages + static_cast<size_t>(idx) * HQ_KV8_PAGE_BYTES;
}

// The new tokens of sequence b: n rows from row0, the first at position first,
// len positions in all.  False (flagged, when `flag`) when the numbers do not
// fit together or the cache; n == 0 is fine and has nothing to do.
struct Kv8Seq {
  int row0, n, first, len;
};
__device__ __forceinline__ bool kv8_seq(const hq_kv8_cache& c, const int32_t* cu, const int32_t* kv_len, int N, int max_new,
                                        int b, bool flag, Kv8Seq& s) {
  const int lo = cu[b], hi = cu[b + 1];
  s.len = kv_len[b];
  s.row0 = lo;
  s.n = 0;
  s.first = s.len;
  uint32_t bad = 0;
  if (lo < 0 || hi < lo || hi > N || hi - lo > max_new || s.len < hi - lo) bad = HQ_DEVERR_ROWS;
  else if (s.len > c.cap) bad = HQ_DEVERR_CAPACITY;
  if (bad) {
    if (flag) kv8_err(c, b, bad);
    return false;
  }
  s.n = hi - lo;
  s.first = s.len - s.n;
  return true;
}

// log2 within 2^-22 (below the normal numbers: -inf), for what needs no more
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Rows of the 16-bit tail enter the value product at a power of two that brings their largest
// value to [2^14, 2^15), as bf16 rows are stored (exact: fp16 rows only go up), and the weight
// takes its inverse: a weight's fp16 range is then spent on the row's own magnitude, and a row
// of zeros has no weight at all.  From the bits of the row's largest magnitude (finite):
__device__ __forceinline__ int kv8_tail_shift(uint32_t top) { return max(0, 29 - max(static_cast<int>(top >> 10), 1)); }
__device__ __forceinline__ float kv8_tail_vscale(float scale, uint32_t top) {  // NaN stays
  if (top == 0) return scale == scale ? 0.f : scale;
  return scale * __uint_as_float(static_cast<uint32_t>(127 - kv8_tail_shift(top)) << 23);
}
// two rows' values times 2^shift, in two steps, for 2^28 is no fp16; tops: their largest magnitudes
struct TailUp {
  __half2 a, b;
  __device__ __forceinline__ explicit TailUp(uint32_t tops) {
    const int x = kv8_tail_shift(tops & 0x7fffu), y = kv8_tail_shift(tops >> 16 & 0x7fffu);
    auto pow2 = [](int k) { return __ushort_as_half(static_cast<unsigned short>((k + 15) << 10)); };
    a = __halves2half2(pow2(min(x, 15)), pow2(min(y, 15)));
    b = __halves2half2(pow2(max(x - 15, 0)), pow2(max(y - 15, 0)));
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const {
    const __half2 r = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&w), a), b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
// larger magnitudes of two pairs
__device__ __forceinline__ uint32_t kv8_top2(uint32_t x, uint32_t y) {
  const __half2 r = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&x)), __habs2(*reinterpret_cast<const __half2*>(&y)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Arguments of the attention kernels (strides in elements).
struct Kv8AttnArgs {
  hq_kv8_cache c;
  const void* q;
  void* out;
  float* lse;
  int64_t q_tok, q_head, o_tok, o_head;
  int Hq, G, N, max_new, window;
  const int32_t* cu;
  const int32_t* kv_len;
  float scale;             // sm_scale * log2 e
  unsigned int* counters;  // of pieces delivered, one for each CTA
  float* parts;            // pieces of tasks that CTAs share
};

// scale of a block from the bits of its largest magnitude (an infinity's or
// NaN's bits are the largest of all); float32 division, as the format says
__device__ __forceinline__ float kv8_scale(uint32_t amax_bits, int fmt) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (amax_bits == 0u) return 1.0f;
  return __fdiv_rn(__uint_as_float(amax_bits), fmt == HQ_KV8_E4M3 ? 448.0f : 127.0f);
}
// The quotients x / scale, each rounded as the division rounds it, by Markstein's
// method (1990): with r = 1 / scale correctly rounded, q = x r and the remainder
// x - q scale (exact in a fused product), q + remainder * r is the correctly rounded
// quotient.  Needs scale, its inverse and the remainders away from the subnormal and
// overflowing ranges: 2^-80 < scale < 2^80 (remainders that underflow then belong to
// quotients that round to zero).  Three operations against a division's dozen.
__device__ __forceinline__ bool kv8_scale_plain(float scale) { return scale > 0x1p-80f && scale < 0x1p80f; }
__device__ __forceinline__ float2 kv8_quotients(float2 x, uint64_t minus_scale2, uint64_t r2) {
  const uint64_t v = f32x2(x.x, x.y), q = f32x2_mul(v, r2);
  return f32x2_split(f32x2_fma(f32x2_fma(q, minus_scale2, v), r2, q));
}
// codes of four quotients (|y| <= 127.5 for int8), lowest byte first
template <int FMT>
__device__ __forceinline__ uint32_t kv8_round4(const float (&y)[4]) {
  if constexpr (FMT == HQ_KV8_E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  } else {
    // |y| < 127.5 (amax / scale is 127 up to rounding): the sum with 1.5 * 2^23 is rounded
    // to an integer, ties to even, and its low byte is the code
    uint32_t z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = __float_as_uint(y[i] + 12582912.0f);
    return prmt(prmt(z[0], z[1], 0x0040u), prmt(z[2], z[3], 0x0040u), 0x5410u);
  }
}
// codes of four values, lowest byte first; `scale` NaN: zeros
template <int FMT>
__device__ __forceinline__ uint32_t kv8_codes4(const float (&x)[4], float scale) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = __fdiv_rn(x[i], scale);
    // a subnormal scale may be far from amax / 127
    if (FMT == HQ_KV8_INT8) y[i] = fminf(fmaxf(y[i], -127.0f), 127.0f);
  }
  return scale == scale ? kv8_round4<FMT>(y) : 0u;
}

// four codes -> two pairs of fp16, exact in both formats
template <int FMT>
__device__ __forceinline__ void kv8_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == HQ_KV8_E4M3) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // a byte with its sign bit flipped, under the exponent of 1024: 1024 + 128 + code
    const uint32_t u = w ^ 0x80808080u;
    lo = hsub2_u(prmt(u, 0x64646464u, 0x4140u), 0x64806480u);
    hi = hsub2_u(prmt(u, 0x64646464u, 0x4342u), 0x64806480u);
  }
}

}  // namespace hq
