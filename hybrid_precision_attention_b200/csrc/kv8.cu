// kv8.cu — writing the 8-bit block cache and reading it back.
//
// A block of 64 positions x 128 values of one (sequence, kv head), K and V
// apart, has one float32 scale: s = amax / 448 (e4m3) or amax / 127 (int8),
// code = round(x / s).  A block is quantised once all its positions are there,
// from their 16-bit values; until then they stand in the tail, which keeps the
// two newest blocks so that up to 64 positions can be taken back.
//
// Both kernels are bound by memory: an append reads each new row once and
// writes its codes once, a read-back the other way round.  16-bit rows pass
// through shared memory as they are: the page's order of values, pairs of tokens
// of one d, is what the transposed 8x8 matrix loads and stores (ldmatrix,
// stmatrix) exchange, so that no element moves by itself.
// Measured (8 kv heads): 5 prompts of 8191 appended in 61 us, 3.9 TB/s (elements moved
// one by one and each divided: 101 us), a token to each of 64 sequences in 8.1 us (a chain of
// look-ups, tail, block); two sequences of 32K read back in 71 us, 5.7 TB/s (115 us), as float32
// in 113 us, 5.9 TB/s; three short ones in 6.0 us.
#include <cuda_runtime.h>

#include <type_traits>

#include "kv8.cuh"

namespace hq {
namespace {

constexpr int T16 = D + 8;  // row stride of a tile of 16-bit elements: 8 rows' 16-byte chunks hit 32 banks
constexpr int TS = D + 4;   // row stride of the staged tile in floats: the V order's accesses (4 rows x 8 columns a step) hit 32 banks
static_assert(D == 128, "the page orders are written for 128");

struct AppendArgs {
  hq_kv8_cache c;
  const void* x[2];
  int64_t tok[2], head[2];
  int N;
  const int32_t* cu;
  const int32_t* kv_len;
};

// four 8x8 matrices of 16-bit elements, transposed: lane l gets of matrix i the
// elements (rows 2 (l % 4), + 1; column l / 4), from the rows that lanes 8 i .. 8 i + 7 address
__device__ __forceinline__ void ldmatrix_t4(uint32_t (&r)[4], const void* row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(row))
               : "memory");
}
// the same places written from those lanes
__device__ __forceinline__ void stmatrix_t4(void* row, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(row)), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
template <class E>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
  if (IsBf16<E>::value) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <class E>
__device__ __forceinline__ uint32_t to_pair(float x, float y) {
  uint32_t w;
  if (IsBf16<E>::value) *reinterpret_cast<__nv_bfloat162*>(&w) = __floats2bfloat162_rn(x, y);
  else *reinterpret_cast<__half2*>(&w) = __floats2half2_rn(x, y);
  return w;
}

// A block whose earlier rows are no numbers of E (they came with calls of another element
// type, or are not finite): every element in float32 from where it lies, a code word of the page at a time,
// amax first.  Rare, and so not tiled.  new_row: the input's row of the block's first
// position, `fresh` rows of it come from the tail.
template <class E, int FMT>
__device__ __noinline__ void append_mixed(const E* new_row, int64_t tok, const uint16_t* tail, const float* scales, int fresh, bool values,
                                          uint8_t* codes, float* scale_out, uint32_t* sh_amax) {
  auto at = [&](int r, int d) {
    return r >= fresh ? to_float(new_row[r * tok + d])
                      : __half2float(__ushort_as_half(tail[values ? HQ_KV8_V_INDEX(r, d) : HQ_KV8_K_INDEX(r, d)])) * scales[r];
  };
  __syncthreads();  // the last reader of sh_amax is done
  if (threadIdx.x == 0) *sh_amax = 0;
  __syncthreads();
  uint32_t top = 0;
  for (int i = threadIdx.x; i < KV8_BLOCK * D; i += 256) top = max(top, __float_as_uint(at(i / D, i % D)) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) atomicMax(sh_amax, top);
  __syncthreads();
  const float scale = kv8_scale(*sh_amax, FMT);
  for (int i = threadIdx.x; i < KV8_BLOCK * D / 4; i += 256) {
    float x[4];  // the word's elements: K four d of a position, V positions r, r + 1, r + 8, r + 9 of one d
    if (values) {
      const int r = i / 512 * 16 + i / 4 % 4 * 2, d = i / 128 % 4 * 32 + (i / 2 % 2) * 16 + (i % 2) * 8 + i / 16 % 8;
      x[0] = at(r, d), x[1] = at(r + 1, d), x[2] = at(r + 8, d), x[3] = at(r + 9, d);
    } else {
      const int r = i / 256 * 8 + i / 16 % 8, d = i / 128 % 2 * 64 + i % 16 * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = at(r, d + j);
    }
    reinterpret_cast<uint32_t*>(codes)[i] = kv8_codes4<FMT>(x, scale);
  }
  if (threadIdx.x == 0) *scale_out = scale;
}

// One CTA per (block that new tokens touch, kv head), K and V: 32 KB of rows in
// flight behind one chain of look-ups.  Sequence b's blocks are CTAs s_b, s_b + 1,
// .. with s_b = cu[b] / 64 + 2 b: n tokens touch at most n / 64 + 2 blocks, so the
// ranges do not overlap and the host needs to know N and B only.
template <class E, int FMT>
__global__ void __launch_bounds__(256, 4) kv8_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ __align__(16) uint16_t tiles[2][KV8_BLOCK * T16];
  __shared__ int sh_b;
  __shared__ Kv8Seq sh_s;
  __shared__ uint32_t sh_amax[2];
  const hq_kv8_cache& c = a.c;
  const int h = blockIdx.y, tid = threadIdx.x, item = blockIdx.x;
  chained();
  if (tid == 0) {
    sh_b = -1;
    sh_amax[0] = sh_amax[1] = 0;
  }
  __syncthreads();
  for (int b = tid; b < c.B; b += 256) {
    // every sequence's numbers are read at once; one CTA says which sequences are skipped
    Kv8Seq s;
    const bool fits = kv8_seq(c, a.cu, a.kv_len, a.N, a.N, b, item == 0 && h == 0, s);
    const int at = s.row0 / KV8_BLOCK + 2 * b;
    if (fits && s.n > 0 && at <= item && item <= at + s.n / KV8_BLOCK + 1) {  // one b at most where cu ascends
      sh_b = b;
      sh_s = s;
    }
  }
  __syncthreads();
  const int b = sh_b;
  if (b < 0) return;
  const Kv8Seq s = sh_s;
  const int first_blk = s.first / KV8_BLOCK, last_blk = (s.len - 1) / KV8_BLOCK;
  const int blk = first_blk + item - (s.row0 / KV8_BLOCK + 2 * b);
  if (blk < first_blk || blk > last_blk) return;
  const size_t bh = static_cast<size_t>(b) * c.Hkv + h;
  const int p0 = blk * KV8_BLOCK, half = blk & 1;
  // position p's row is src + p * tok
  auto source = [&](int which) {
    return static_cast<const E*>(a.x[which]) + static_cast<int64_t>(s.row0 - s.first) * a.tok[which] + h * a.head[which];
  };
  auto tail_of = [&](int which) { return (which ? c.tail_v : c.tail_k) + bh * HQ_KV8_TAIL * D; };
  auto scales_of = [&](int which) { return c.tail_scale + (bh * 2 + which) * HQ_KV8_TAIL; };

  if (p0 + KV8_BLOCK <= s.len) {
    // the block is complete: its rows into the tiles, new ones from the input,
    // earlier ones from the tail
    const long long idx = kv8_page_index(c, bh, blk);
    uint4 v[2][4];
    int lost = 0;  // earlier elements that E does not hold
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const E* src = source(which);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int e = it * 256 + tid, p = p0 + e / 16, d = e % 16 * 8;
        if (p >= s.first) {
          v[which][it] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(p) * a.tok[which] + d);
        } else {
          const int r = p - p0;
          const float sc = scales_of(which)[half * KV8_BLOCK + r];
          const uint16_t* t = tail_of(which) + half * KV8_BLOCK * D;
          E x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[i] = from_float<E>(__half2float(__ushort_as_half(t[which ? HQ_KV8_V_INDEX(r, d + i) : HQ_KV8_K_INDEX(r, d + i)])) * sc);
          // at another scale than 1 the row came as bf16, at 1 as fp16, or it is one for which both say the same
          if (!IsBf16<E>::value) {
            lost |= sc != 1.0f;
          } else if (sc == 1.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              lost |= to_float(x[i]) != __half2float(__ushort_as_half(t[which ? HQ_KV8_V_INDEX(r, d + i) : HQ_KV8_K_INDEX(r, d + i)]));
          }
          v[which][it] = *reinterpret_cast<const uint4*>(x);
        }
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      // magnitudes compare as integers: the 15 bits of each half
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int e = it * 256 + tid;
        const uint32_t w[4] = {v[which][it].x, v[which][it].y, v[which][it].z, v[which][it].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi = max(hi, w[i] & 0x7fff0000u);
          lo = max(lo, w[i] & 0x7fffu);
        }
        *reinterpret_cast<uint4*>(tiles[which] + e / 16 * T16 + e % 16 * 8) = v[which][it];
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, max(hi >> 16, lo));
      if ((tid & 31) == 0) atomicMax(&sh_amax[which], top);
    }
    const bool mixed = __syncthreads_or(lost);
    if (idx < 0) {
      if (tid == 0) kv8_err(c, b, HQ_DEVERR_PAGE);
    } else if (mixed) {
      uint8_t* page = c.pages + static_cast<size_t>(idx) * HQ_KV8_PAGE_BYTES;
#pragma unroll 1
      for (int which = 0; which < 2; ++which)
        append_mixed<E, FMT>(source(which) + static_cast<int64_t>(p0) * a.tok[which], a.tok[which],
                             tail_of(which) + half * KV8_BLOCK * D, scales_of(which) + half * KV8_BLOCK, s.first - p0, which,
                             page + (which ? HQ_KV8_V : 0), reinterpret_cast<float*>(page + (which ? HQ_KV8_VSCALE : HQ_KV8_KSCALE)),
                             &sh_amax[which]);
    } else {
      uint8_t* page = c.pages + static_cast<size_t>(idx) * HQ_KV8_PAGE_BYTES;
      const int lane = tid & 31;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const float scale = kv8_scale(__float_as_uint(pair_of<E>(sh_amax[which]).x), FMT);
        const bool plain = kv8_scale_plain(scale);
        const float r = 1.0f / scale;
        const uint64_t minus2 = f32x2(-scale, -scale), r2 = f32x2(r, r);
#pragma unroll
        for (int it = 0; it < 2; ++it) {
          const int e = it * 256 + tid;  // 16-byte chunk of the page's codes
          uint32_t x[8], w[4];           // its elements: two of a word, four of a code word
          if (which) {
            // tokens 16 tt .. + 15, d 32 dq ..: matrices of 8 tokens x 8 d
            const int tt = e / 128, dq = e / 32 % 4;
            const uint16_t* row = tiles[1] + (tt * 16 + (lane >> 3 & 1) * 8 + (lane & 7)) * T16 + dq * 32 + (lane >> 4) * 8;
            uint32_t m[4];
            ldmatrix_t4(m, row);         // (tokens 0-7, 8-15) of d 0-7, then of d 8-15
            x[0] = m[0], x[1] = m[1], x[2] = m[2], x[3] = m[3];
            ldmatrix_t4(m, row + 16);
            x[4] = m[0], x[5] = m[1], x[6] = m[2], x[7] = m[3];
          } else {
            const uint4* row = reinterpret_cast<const uint4*>(tiles[0] + (e / 64 * 8 + e / 4 % 8) * T16 + e / 32 % 2 * 64 + (e & 3) * 16);
            *reinterpret_cast<uint4*>(x) = row[0];
            *reinterpret_cast<uint4*>(x + 4) = row[1];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = pair_of<E>(x[2 * i]), z = pair_of<E>(x[2 * i + 1]);
            if (plain) {
              const float2 qy = kv8_quotients(y, minus2, r2), qz = kv8_quotients(z, minus2, r2);
              const float q[4] = {qy.x, qy.y, qz.x, qz.y};
              w[i] = kv8_round4<FMT>(q);
            } else {
              const float q[4] = {y.x, y.y, z.x, z.y};
              w[i] = kv8_codes4<FMT>(q, scale);
            }
          }
          reinterpret_cast<uint4*>(page + (which ? HQ_KV8_V : 0))[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (tid == 0) *reinterpret_cast<float*>(page + (which ? HQ_KV8_VSCALE : HQ_KV8_KSCALE)) = scale;
      }
    }
  }
  // The tail's half of this block's parity is written by one CTA alone, the
  // first touched block of that parity: it is the only one that may have read
  // earlier rows there (above; the barrier orders the two), and it writes the
  // new rows of the last touched block of that parity.
  if (blk > first_blk + 1) return;
  __syncthreads();
  const int t0 = (last_blk - ((last_blk - blk) & 1)) * KV8_BLOCK;
  const int warp = tid / 32, lane = tid % 32;
  const int begin = max(t0, s.first), rows = min(t0 + KV8_BLOCK, s.len) - begin;
  for (int i0 = warp; i0 < 2 * rows; i0 += 4 * 8) {  // K and V rows in turn, four of a warp in flight
    uint2 in[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + 8 * q, which = i & 1;
      if (i < 2 * rows)
        in[q] = *reinterpret_cast<const uint2*>(source(which) + static_cast<int64_t>(begin + i / 2) * a.tok[which] + lane * 4);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + 8 * q, which = i & 1, p = begin + i / 2;
      if (i >= 2 * rows) break;
      E e[4];
      *reinterpret_cast<uint2*>(e) = in[q];
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = max(amax, __float_as_uint(to_float(e[j])) & 0x7fffffffu);
      amax = __reduce_max_sync(0xffffffffu, amax);
      float sc = 1.0f;
      if (amax >= 0x7f800000u) {
        sc = __uint_as_float(0x7fc00000u);
      } else if (IsBf16<E>::value && amax != 0) {
        // the power of two that brings amax to [2^14, 2^15), itself a normal number
        const int ex = max(static_cast<int>(amax >> 23) - 127 - 14, -126);
        sc = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
      }
      uint16_t* t = tail_of(which) + half * KV8_BLOCK * D;
      const int r = p % KV8_BLOCK;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = lane * 4 + j;
        // the division by a power of two is exact, the rounding is to fp16 (exact for fp16 rows)
        const __half y = sc == sc ? __float2half_rn(to_float(e[j]) / sc) : __float2half_rn(0.f);
        t[which ? HQ_KV8_V_INDEX(r, d) : HQ_KV8_K_INDEX(r, d)] = __half_as_ushort(y);
      }
      if (lane == 0) scales_of(which)[p % HQ_KV8_TAIL] = sc;
    }
  }
}

struct ReadArgs {
  hq_kv8_cache c;
  const int32_t* kv_len;
  int start, n, zero_rest;
  void* out[2];
  int64_t batch, head, tok;
};

// One CTA per (block, kv head and K or V, sequence): the page's 16-byte chunks
// are dequantised into a row-major tile and its rows written out.
template <class E, int FMT>
__global__ void __launch_bounds__(256) kv8_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int STR = sizeof(E) == 2 ? T16 : TS;
  __shared__ __align__(16) E tile[KV8_BLOCK * STR];
  const hq_kv8_cache& c = a.c;
  const int h = blockIdx.y >> 1, which = blockIdx.y & 1, b = blockIdx.z, tid = threadIdx.x;
  const int blk = a.start / KV8_BLOCK + blockIdx.x, p0 = blk * KV8_BLOCK;
  int len = a.kv_len[b];
  if (len > c.cap || len < 0) {
    if (tid == 0) kv8_err(c, b, len < 0 ? HQ_DEVERR_ROWS : HQ_DEVERR_CAPACITY);
    len = 0;
  }
  const size_t bh = static_cast<size_t>(b) * c.Hkv + h;
  if (p0 + KV8_BLOCK <= len) {
    const uint8_t* page = kv8_page(c, bh, blk);
    const float scale = *reinterpret_cast<const float*>(page + (which ? HQ_KV8_VSCALE : HQ_KV8_KSCALE));
    uint4 u[2];
#pragma unroll
    for (int it = 0; it < 2; ++it) u[it] = reinterpret_cast<const uint4*>(page + (which ? HQ_KV8_V : 0))[it * 256 + tid];
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int e = it * 256 + tid, lane = tid & 31;
      const uint32_t w[4] = {u[it].x, u[it].y, u[it].z, u[it].w};
      float x[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t p, q;
        kv8_half4<FMT>(w[i], p, q);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p)), g = __half22float2(*reinterpret_cast<const __half2*>(&q));
        x[4 * i] = f.x * scale;
        x[4 * i + 1] = f.y * scale;
        x[4 * i + 2] = g.x * scale;
        x[4 * i + 3] = g.y * scale;
      }
      // K: 16 d of one token; V: tokens r, r + 1, r + 8, r + 9 of d, d + 8, d + 16, d + 24
      const int rk = e / 64 * 8 + e / 4 % 8, dk = e / 32 % 2 * 64 + (e & 3) * 16;
      const int tt = e / 128, dq = e / 32 % 4;
      if constexpr (sizeof(E) == 2) {
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = to_pair<E>(x[2 * i], x[2 * i + 1]);
        if (which) {
          E* row = tile + (tt * 16 + (lane >> 3 & 1) * 8 + (lane & 7)) * STR + dq * 32 + (lane >> 4) * 8;
          const uint32_t m0[4] = {y[0], y[1], y[2], y[3]}, m1[4] = {y[4], y[5], y[6], y[7]};
          stmatrix_t4(row, m0);
          stmatrix_t4(row + 16, m1);
        } else {
          uint4* row = reinterpret_cast<uint4*>(tile + rk * STR + dk);
          row[0] = make_uint4(y[0], y[1], y[2], y[3]);
          row[1] = make_uint4(y[4], y[5], y[6], y[7]);
        }
      } else if (which) {
        const int r = tt * 16 + (e & 3) * 2, d = dq * 32 + e / 4 % 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          E* t = tile + r * STR + d + 8 * i;
          t[0] = x[4 * i];
          t[STR] = x[4 * i + 1];
          t[8 * STR] = x[4 * i + 2];
          t[9 * STR] = x[4 * i + 3];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(tile + rk * STR + dk + 4 * i) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
    }
  } else if (p0 < len) {
    const uint16_t* t = (which ? c.tail_v : c.tail_k) + (bh * 2 + (blk & 1)) * KV8_BLOCK * D;
    const float* sc = c.tail_scale + (bh * 2 + which) * HQ_KV8_TAIL + (blk & 1) * KV8_BLOCK;
    for (int e = tid; e < (len - p0) * D; e += 256) {
      const int r = e / D, d = e % D;
      tile[r * STR + d] = from_float<E>(__half2float(__ushort_as_half(t[which ? HQ_KV8_V_INDEX(r, d) : HQ_KV8_K_INDEX(r, d)])) * sc[r]);
    }
  }
  __syncthreads();
  E* out = static_cast<E*>(a.out[which]) + b * a.batch + h * a.head;
  constexpr int V = 16 / sizeof(E);
#pragma unroll
  for (int it = 0; it < KV8_BLOCK * D / V / 256; ++it) {
    const int e = it * 256 + tid, r = e / (D / V), d = e % (D / V) * V, p = p0 + r;
    if (p < a.start || p >= a.start + a.n || (p >= len && !a.zero_rest)) continue;
    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(p - a.start) * a.tok + d) =
        p < len ? *reinterpret_cast<const uint4*>(tile + r * STR + d) : make_uint4(0u, 0u, 0u, 0u);
  }
}

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

hq_status kv8_validate(const hq_kv8_cache* c) {
  if (!c) return HQ_ERR_INVALID;
  if (c->D != HQ_HEAD_DIM) return HQ_ERR_UNSUPPORTED;
  if (c->B <= 0 || c->Hkv <= 0 || c->cap <= 0 || c->cap % 128 != 0) return HQ_ERR_INVALID;
  if (c->fmt != HQ_KV8_E4M3 && c->fmt != HQ_KV8_INT8) return HQ_ERR_INVALID;
  if (c->B > HQ_KV8_MAX_BATCH || c->Hkv > HQ_KV8_MAX_HEADS) return HQ_ERR_UNSUPPORTED;
  if (!aligned16(c->pages) || !aligned16(c->tail_k) || !aligned16(c->tail_v) || !aligned16(c->tail_scale) || !aligned4(c->err))
    return HQ_ERR_INVALID;
  if (c->page_table != nullptr && (!aligned4(c->page_table) || c->n_pages < 1)) return HQ_ERR_INVALID;
  return HQ_OK;
}

}  // namespace hq

extern "C" {

hq_status hq_kv8_validate(const hq_kv8_cache* c) { return hq::kv8_validate(c); }

hq_status hq_kv8_append(const hq_kv8_cache* c, int32_t dtype, const void* k, int64_t k_tok, int64_t k_head, const void* v,
                        int64_t v_tok, int64_t v_head, int32_t N, const int32_t* cu, const int32_t* kv_len,
                        hq_stream_t stream) {
  const hq_status st = hq::kv8_validate(c);
  if (st != HQ_OK) return st;
  if ((dtype != HQ_F16 && dtype != HQ_BF16) || N < 0 || !hq::aligned4(cu) || !hq::aligned4(kv_len)) return HQ_ERR_INVALID;
  if (N == 0) return HQ_OK;
  // the stride of a dimension of one is never used, whatever it says
  if (N == 1) k_tok = v_tok = 0;
  if (c->Hkv == 1) k_head = v_head = 0;
  if (!hq::aligned16(k) || !hq::aligned16(v) || (k_tok | k_head | v_tok | v_head) % 8) return HQ_ERR_INVALID;
  hq::AppendArgs a = {*c, {k, v}, {k_tok, v_tok}, {k_head, v_head}, N, cu, kv_len};
  const dim3 grid(static_cast<unsigned>(N) / hq::KV8_BLOCK + 2u * c->B, c->Hkv);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) { return hq::cuda_status(hq::launch_chained(kernel, grid, 256, 0, s, a), "kv8 append launch"); };
  const bool f8 = c->fmt == HQ_KV8_E4M3;
  if (dtype == HQ_F16)
    return f8 ? go(hq::kv8_append_kernel<__half, HQ_KV8_E4M3>) : go(hq::kv8_append_kernel<__half, HQ_KV8_INT8>);
  return f8 ? go(hq::kv8_append_kernel<__nv_bfloat16, HQ_KV8_E4M3>) : go(hq::kv8_append_kernel<__nv_bfloat16, HQ_KV8_INT8>);
}

hq_status hq_kv8_read(const hq_kv8_cache* c, int32_t dtype, const int32_t* kv_len, int32_t start, int32_t n, void* k_out,
                      void* v_out, int64_t o_batch, int64_t o_head, int64_t o_tok, int32_t zero_rest, hq_stream_t stream) {
  const hq_status st = hq::kv8_validate(c);
  if (st != HQ_OK) return st;
  if (dtype < HQ_F16 || dtype > HQ_F32 || start < 0 || n < 0 || !hq::aligned4(kv_len)) return HQ_ERR_INVALID;
  if (n == 0) return HQ_OK;
  if (start > c->cap || n > c->cap - start) return HQ_ERR_CAPACITY;
  if (c->B == 1) o_batch = 0;
  if (c->Hkv == 1) o_head = 0;
  if (n == 1) o_tok = 0;
  if (!hq::aligned16(k_out) || !hq::aligned16(v_out) || (o_batch | o_head | o_tok) % 8) return HQ_ERR_INVALID;
  hq::ReadArgs a = {*c, kv_len, start, n, zero_rest, {k_out, v_out}, o_batch, o_head, o_tok};
  const dim3 grid((start + n - 1) / hq::KV8_BLOCK - start / hq::KV8_BLOCK + 1, 2 * c->Hkv, c->B);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // a plain launch: with a chained one the read of 8 short sequences took 6.9 us, not 6.0
  auto go = [&](auto kernel) {
    kernel<<<grid, 256, 0, s>>>(a);
    return hq::cuda_status(cudaGetLastError(), "kv8 read launch");
  };
  auto form = [&](auto fmt) {
    constexpr int F = decltype(fmt)::value;
    if (dtype == HQ_F16) return go(hq::kv8_read_kernel<__half, F>);
    if (dtype == HQ_BF16) return go(hq::kv8_read_kernel<__nv_bfloat16, F>);
    return go(hq::kv8_read_kernel<float, F>);
  };
  if (c->fmt == HQ_KV8_E4M3) return form(std::integral_constant<int, HQ_KV8_E4M3>{});
  return form(std::integral_constant<int, HQ_KV8_INT8>{});
}

}  // extern "C"
