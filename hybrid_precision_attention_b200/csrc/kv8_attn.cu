// kv8_attn.cu — attention of the newest tokens over the 8-bit block cache.
//
// o_r = sum_j p_rj v_j, p = softmax_j(q_r . k_j * sm_scale), keys and values at
// code * scale (one scale per block of 64), the incomplete last block in 16
// bits.  Bound by memory: 256 bytes of codes per position and kv head; every
// page is brought on chip once, by one bulk copy, and its codes meet the tensor
// cores as fp16 (exact for e4m3 and int8; the scales go to the scores and the
// weights in float32).
//
// The rows of a kv head (its G query heads x the sequence's n new tokens, row
// r = i G + g) are taken 8 NB at a time as the N side of m16n8k16 products:
//   S^T [16 tokens x 8 NB rows] = K [16 x 128] Q^T       (A = codes of 16 tokens)
//   O^T [128 x 8 NB rows]      += V^T [128 x 16] P^T     (A = codes of 16 tokens)
// so that 8 rows waste nothing of the product, where rows on the M side would
// waste half of it.  The page's element orders are the A operands' own: a
// thread's 16-byte load is its operand for four steps, with no conflict and no
// shuffle.  P^T comes from S^T by a register transpose (movmatrix).
//
// Work: the tasks (sequence, kv head, 8 NB rows) have their blocks laid end to
// end and cut into gridDim equal runs.  A task that one CTA holds whole is
// finished there; the pieces of the others go to the workspace and the CTA that
// delivers a task's last piece joins them in order, so that results do not
// depend on timing.  Within a CTA a producer warp keeps a ring of pages in
// flight and NG groups of 4 warps take every NG-th block, 16 tokens a warp, each
// warp with its own running maximum, sum and accumulators.
//
// Two running references per row, both powers of two exponents: m, the maximum
// score, for the sum of weights; E, the maximum of score + log2(value scale),
// for the accumulators, whose weights p * vscale enter the product as fp16 at
// 2^14 * 2^(s + log2 vscale - E): the largest is 2^14, and the smallest normal
// one is 2^-28 of it, whatever the ratios of the blocks' scales.
#include <cuda_runtime.h>

#include <type_traits>

#include "kv8.cuh"

namespace hq {
namespace {

constexpr float P_BIAS = 14.0f;  // log2 of the largest fp16 weight
constexpr int OS = D + 4;        // row stride (floats) of accumulators in shared memory: 4 rows of a store step 8 banks apart

template <int NB, int NG>
struct Cfg {
  static constexpr int R = 8 * NB;            // rows of a task
  static constexpr int WARPS = 4 * NG;        // consumers
  static constexpr int THREADS = WARPS * 32 + 32;
  static constexpr int OBUF = WARPS * R * OS * 4;
  static constexpr int RED = WARPS * R * 16;  // (m, E, l) of each warp's rows
  static constexpr int FIXED = OBUF + RED + 256;
  static constexpr int STAGE_MAX = 12;
};

struct AttnArgs {
  hq_kv8_cache c;
  const void* q;
  void* out;
  float* lse;
  int64_t q_tok, q_head, o_tok, o_head;
  int Hq, G, N, max_new, window, groups;  // groups: tasks of a (sequence, kv head)
  int stages;
  const int32_t* cu;
  const int32_t* kv_len;
  float scale;  // sm_scale * log2 e
  unsigned int* counters;
  float* parts;
};

// blocks of sequence s that its queries see: [begin, end)
__device__ __forceinline__ void seq_blocks(const Kv8Seq& s, int window, int& begin, int& end) {
  begin = window > 0 ? max(0, s.first + 1 - window) / KV8_BLOCK : 0;
  end = s.n > 0 ? (s.len + KV8_BLOCK - 1) / KV8_BLOCK : begin;
}

__device__ __forceinline__ float log2_acc(float x) { return log2f(x); }

// Bounded wait on a page of the ring; a copy that does not land within about a
// second sets the sequence's error bit and ends the CTA's work.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, int32_t* err, volatile int* stop) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if (global_ns() - t0 > 1000000000ull) {
      atomicOr(reinterpret_cast<unsigned int*>(err), HQ_DEVERR_TIMEOUT);
      *stop = 1;
      return false;
    }
  }
  return true;
}

template <class E, int FMT, int NB, int NG>
__global__ void __launch_bounds__(Cfg<NB, NG>::THREADS, 1) kv8_attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<NB, NG>;
  constexpr int R = C::R, CT = C::WARPS * 32;
  extern __shared__ __align__(128) uint8_t sm[];
  float* obuf = reinterpret_cast<float*>(sm);                    // [warp][row][OS]
  float4* red = reinterpret_cast<float4*>(sm + C::OBUF);         // [warp][row] (m, E, l, -)
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OBUF + C::RED);
  uint64_t* empty = full + C::STAGE_MAX;
  int* flags = reinterpret_cast<int*>(empty + C::STAGE_MAX);     // stop, last, total lo, hi
  int* prefix = reinterpret_cast<int*>(sm + C::FIXED);           // blocks of the sequences before b (per task)
  const int B = a.c.B;
  uint8_t* ring = sm + C::FIXED + ((B + 1) * 4 + 127) / 128 * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const hq_kv8_cache& c = a.c;

  // ---------------------------------------------------------------- plan
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 4);
    }
    fence_mbar_init();
    flags[0] = 0;
  }
  if (warp == 0) {
    int sum = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      int n = 0;
      if (b0 + lane < B) {
        Kv8Seq s;
        kv8_seq(c, a.cu, a.kv_len, a.N, a.max_new, b0 + lane, blockIdx.x == 0, s);
        int begin, end;
        seq_blocks(s, a.window, begin, end);
        n = end - begin;
      }
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < B) prefix[b0 + lane] = sum + x - n;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) prefix[B] = sum;
  }
  __syncthreads();
  const int per_seq = c.Hkv * a.groups;  // tasks of a sequence
  const long long total = static_cast<long long>(prefix[B]) * per_seq;
  const long long parts = min(total, static_cast<long long>(gridDim.x));  // CTAs with work: each has a block at least
  if (blockIdx.x >= parts) return;
  const long long u0 = total * blockIdx.x / parts, u1 = total * (blockIdx.x + 1) / parts;
  volatile int* stop = flags;

  // Walks the CTA's run task by task: [t0, t1) of the task's blocks are ours.
  struct Task {
    int b, h, grp, begin, blocks, t0, t1;
    Kv8Seq s;
  };
  auto task_at = [&](long long u, Task& k) {
    const long long want = u / per_seq;  // the sequence holding unit u: prefix[b] <= u / per_seq < prefix[b + 1]
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= want) lo = mid; else hi = mid;
    }
    k.b = lo;
    kv8_seq(c, a.cu, a.kv_len, a.N, a.max_new, lo, false, k.s);
    int end;
    seq_blocks(k.s, a.window, k.begin, end);
    k.blocks = end - k.begin;
    const long long rel = u - static_cast<long long>(prefix[lo]) * per_seq;
    const int task = static_cast<int>(rel / k.blocks);
    k.h = task / a.groups;
    k.grp = task - k.h * a.groups;
    k.t0 = static_cast<int>(rel - static_cast<long long>(task) * k.blocks);
    k.t1 = static_cast<int>(min(static_cast<long long>(k.blocks), k.t0 + (u1 - u)));
  };

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int n = 0;
      bool ok = true;
      for (long long u = u0; ok && u < u1;) {
        Task k;
        task_at(u, k);
        const size_t bh = static_cast<size_t>(k.b) * c.Hkv + k.h;
        for (int t = k.t0; ok && t < k.t1; ++t) {
          const int blk = k.begin + t;
          if ((blk + 1) * KV8_BLOCK > k.s.len) continue;  // the tail is read where it lies
          const int st = n % a.stages;
          const uint8_t* page = kv8_page(c, bh, blk);
          if (n >= a.stages) ok = ring_wait(empty + st, (n / a.stages - 1) & 1, c.err + k.b, stop);
          if (!ok) break;
          mbar_arrive_expect_tx(full + st, KV8_COPY);
          bulk_g2s(ring + st * HQ_KV8_PAGE_BYTES, page, KV8_COPY, full + st);
          ++n;
        }
        u += k.t1 - k.t0;
      }
      // no copy may be in flight when the CTA's shared memory is given up; the
      // consumers have waited for all of them unless they stopped early
      if (*stop) {
        int never = 0;
        for (int i = max(0, n - a.stages); i < n; ++i) ring_wait(full + i % a.stages, (i / a.stages) & 1, c.err, &never);
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int grp4 = warp >> 2, tt = warp & 3;  // group of 4 warps; the warp's 16 tokens of a block
  const int g = lane >> 2, t4 = lane & 3;
  int n_ring = 0, turn = 0;  // pages taken from the ring, blocks seen: by all groups together
  bool ok = true;
  for (long long u = u0; u < u1;) {
    Task k;
    task_at(u, k);
    const size_t bh = static_cast<size_t>(k.b) * c.Hkv + k.h;
    const int row0 = k.grp * R, rows = k.s.n * a.G;

    // query rows as B operands: lane (g, t4) holds row g (+ 8 nb), elements
    // 64 j + 16 t4 + 4 u + {0..3} at step 4 j + u, the elements that the K codes'
    // 16-byte chunk t4 of half j gives at that step
    uint32_t qf[NB][16];
    float qs[NB][2];   // multiplier of the scores of rows 2 t4, 2 t4 + 1
    int qp[NB][2];     // their positions, -1: no such row
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = row0 + 8 * nb + g;
      float mul = 1.0f;
      uint4 v[4] = {};
      if (r < rows) {
        const E* p = static_cast<const E*>(a.q) + static_cast<int64_t>(k.s.row0 + r / a.G) * a.q_tok +
                     static_cast<int64_t>(k.h * a.G + r % a.G) * a.q_head + 16 * t4;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[2 * j] = *reinterpret_cast<const uint4*>(p + 64 * j);
          v[2 * j + 1] = *reinterpret_cast<const uint4*>(p + 64 * j + 8);
        }
      }
      const E* e = reinterpret_cast<const E*>(v);
      if (IsBf16<E>::value) {
        // bf16 rows become fp16 at a power of two that brings their largest value to [2^14, 2^15)
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(to_float(e[i])) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float inv = 1.0f;
        if (m != 0 && m < 0x7f800000u) {
          const int ex = max(static_cast<int>(m >> 23) - 127 - 14, -126);  // at most 113
          mul = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
          inv = ex == -126 ? 0x1p126f : __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) qf[nb][i] = pack_f16x2(to_float(e[2 * i]) * inv, to_float(e[2 * i + 1]) * inv);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) qf[nb][i] = reinterpret_cast<const uint32_t*>(v)[i];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qs[nb][i] = __shfl_sync(0xffffffffu, mul, (2 * t4 + i) * 4) * a.scale;
        const int rr = row0 + 8 * nb + 2 * t4 + i;
        qp[nb][i] = rr < rows ? k.s.first + rr / a.G : -1;
      }
    }

    float o[NB][8][4];
    float m_run[NB][2], e_run[NB][2], l_run[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][mt][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) m_run[nb][i] = e_run[nb][i] = -INFINITY, l_run[nb][i] = 0.f;
    }

    // one 16-token tile: kf, vf give the A operands of step s / output rows 16 mt
    // .. 16 mt + 15; ks, vs the scales of tokens g, g + 8; pos the first token's position
    auto tile = [&](auto kf, auto vf, const float (&ks)[2], const float (&vs)[2], float vtop, int pos) {
      float sc[NB][4];
      {
        float s2[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[nb][i] = s2[nb][i] = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          uint32_t f[4];
          kf(s, f);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(s & 1 ? s2[nb] : sc[nb], f[0], f[1], f[2], f[3], qf[nb][2 * s], qf[nb][2 * s + 1]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[nb][i] += s2[nb][i];
      }
      const float lv = log2_acc(vtop);
      uint32_t pf[NB][2];
      bool moved = false;
      float ao[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // rows 2 t4 + i
          const float mul = qs[nb][i];
          const int d0 = qp[nb][i] - (pos + g), d1 = d0 - 8;  // how far the tokens lie behind the query
          const bool in0 = d0 >= 0 && (a.window <= 0 || d0 < a.window), in1 = d1 >= 0 && (a.window <= 0 || d1 < a.window);
          const float s0 = in0 ? sc[nb][i] * (mul * ks[0]) : -INFINITY;
          const float s1 = in1 ? sc[nb][2 + i] * (mul * ks[1]) : -INFINITY;
          float mt = fmaxf(s0, s1);
          mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
          mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
          mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
          const float m_new = fmaxf(m_run[nb][i], mt), e_new = fmaxf(e_run[nb][i], mt + lv);
          const float mb = m_new == -INFINITY ? 0.f : m_new, eb = e_new == -INFINITY ? 0.f : e_new;
          const float al = ex2(m_run[nb][i] - mb);
          ao[nb][i] = ex2(e_run[nb][i] - eb);
          moved |= e_new > e_run[nb][i];
          m_run[nb][i] = m_new;
          e_run[nb][i] = e_new;
          const float p0 = ex2(s0 - mb), p1 = ex2(s1 - mb);
          l_run[nb][i] = l_run[nb][i] * al + (p0 + p1);
          // p * vscale at 2^14 / 2^E; the exponent is bounded so that a weight that
          // underflowed to 0 stays 0 beside a far larger earlier score
          const float f = ex2(fminf(mb - eb + P_BIAS + lv, 100.f));
          p[i] = in0 ? p0 * (f * vs[0]) : 0.f;
          p[2 + i] = in1 ? p1 * (f * vs[1]) : 0.f;
        }
        pf[nb][0] = movmatrix_t(pack_f16x2(p[0], p[1]));
        pf[nb][1] = movmatrix_t(pack_f16x2(p[2], p[3]));
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nb][mt][i] *= ao[nb][i & 1];
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        uint32_t f[4];
        vf(mt, f);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][mt], f[0], f[1], f[2], f[3], pf[nb][0], pf[nb][1]);
      }
    };

    for (int t = k.t0; t < k.t1; ++t) {
      const int blk = k.begin + t, p0 = blk * KV8_BLOCK;
      const bool mine = turn % NG == grp4;
      ++turn;
      if (p0 + KV8_BLOCK <= k.s.len) {
        const int st = n_ring % a.stages, ph = (n_ring / a.stages) & 1;
        ++n_ring;
        if (!mine || !ok) continue;
        ok = ring_wait(full + st, ph, c.err + k.b, stop);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        const uint8_t* page = ring + st * HQ_KV8_PAGE_BYTES;
        const float2 sc = *reinterpret_cast<const float2*>(page + HQ_KV8_KSCALE);
        uint4 kw[4], vw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kw[i] = reinterpret_cast<const uint4*>(page + tt * 2048 + i * 512)[lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) vw[i] = reinterpret_cast<const uint4*>(page + HQ_KV8_V + tt * 2048 + i * 512)[lane];
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + st);
        auto word = [](const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; };
        const float ks[2] = {sc.x, sc.x}, one[2] = {1.f, 1.f};
        tile(
            [&](int s, uint32_t (&f)[4]) {
              // chunk (token half a, d half j) = 2 a + j; word s % 4 of it
              kv8_half4<FMT>(word(kw[s >> 2], s & 3), f[0], f[2]);
              kv8_half4<FMT>(word(kw[2 + (s >> 2)], s & 3), f[1], f[3]);
            },
            [&](int mt, uint32_t (&f)[4]) {
              kv8_half4<FMT>(word(vw[mt >> 1], (mt & 1) * 2), f[0], f[2]);
              kv8_half4<FMT>(word(vw[mt >> 1], (mt & 1) * 2 + 1), f[1], f[3]);
            },
            ks, one, sc.y, p0 + tt * 16);
      } else {
        // the incomplete block, in 16 bits: rows past the length hold finite
        // values of earlier blocks or zeros and are masked
        if (!mine || p0 + tt * 16 >= k.s.len) continue;
        const int half = blk & 1;
        const uint4* tk = reinterpret_cast<const uint4*>(c.tail_k + (bh * 2 + half) * KV8_BLOCK * D + tt * 2048);
        const uint4* tv = reinterpret_cast<const uint4*>(c.tail_v + (bh * 2 + half) * KV8_BLOCK * D + tt * 2048);
        const float* ts = c.tail_scale + bh * 2 * HQ_KV8_TAIL + half * KV8_BLOCK + tt * 16 + g;
        const bool in0 = p0 + tt * 16 + g < k.s.len, in1 = p0 + tt * 16 + g + 8 < k.s.len;
        const float ks[2] = {in0 ? ts[0] : 1.f, in1 ? ts[8] : 1.f};
        float vs[2] = {in0 ? ts[HQ_KV8_TAIL] : 0.f, in1 ? ts[HQ_KV8_TAIL + 8] : 0.f};
        float vtop = fmaxf(vs[0], vs[1]);  // ignores NaN
        vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, 4));
        vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, 8));
        vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, 16));
        if (!(vtop > 0.f)) vtop = 1.f;
        vs[0] = vs[0] / vtop;
        vs[1] = vs[1] / vtop;
        uint32_t kw[4][8], vw[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *reinterpret_cast<uint4*>(&kw[i][0]) = tk[(i * 32 + lane) * 2];
          *reinterpret_cast<uint4*>(&kw[i][4]) = tk[(i * 32 + lane) * 2 + 1];
          *reinterpret_cast<uint4*>(&vw[i][0]) = tv[(i * 32 + lane) * 2];
          *reinterpret_cast<uint4*>(&vw[i][4]) = tv[(i * 32 + lane) * 2 + 1];
        }
        tile(
            [&](int s, uint32_t (&f)[4]) {
              f[0] = kw[s >> 2][(s & 3) * 2];
              f[2] = kw[s >> 2][(s & 3) * 2 + 1];
              f[1] = kw[2 + (s >> 2)][(s & 3) * 2];
              f[3] = kw[2 + (s >> 2)][(s & 3) * 2 + 1];
            },
            [&](int mt, uint32_t (&f)[4]) {
              const int w = (mt & 1) * 4;
              f[0] = vw[mt >> 1][w];
              f[2] = vw[mt >> 1][w + 1];
              f[1] = vw[mt >> 1][w + 2];
              f[3] = vw[mt >> 1][w + 3];
            },
            ks, vs, vtop, p0 + tt * 16);
      }
    }

    // ------------------------------------------------------------ the CTA's piece of the task
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = l_run[nb][i];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) red[warp * R + 8 * nb + 2 * t4 + i] = make_float4(m_run[nb][i], e_run[nb][i], l, 0.f);
      }
    asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory");
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * nb + 2 * t4 + i;
        float e = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) e = fmaxf(e, red[w * R + r].y);
        const float f = e == -INFINITY ? 1.f : ex2(e_run[nb][i] - e);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          obuf[(warp * R + r) * OS + mt * 16 + g] = o[nb][mt][i] * f;
          obuf[(warp * R + r) * OS + mt * 16 + g + 8] = o[nb][mt][2 + i] * f;
        }
      }
    // this thread's outputs: rows warp, warp + WARPS, .., elements 4 lane .. 4 lane + 3
    constexpr int RPW = (R + C::WARPS - 1) / C::WARPS;
    float rm[RPW], re[RPW], rl[RPW];
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int r = warp + i * C::WARPS;
      rm[i] = re[i] = -INFINITY;
      rl[i] = 0.f;
      if (r < R) {
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float4 x = red[w * R + r];
          rm[i] = fmaxf(rm[i], x.x);
          re[i] = fmaxf(re[i], x.y);
        }
        const float mb = rm[i] == -INFINITY ? 0.f : rm[i];
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float4 x = red[w * R + r];
          rl[i] += x.z * ex2(x.x - mb);
        }
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory");
    float4 acc[RPW];
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int r = warp + i * C::WARPS;
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < R) {
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(obuf + (w * R + r) * OS + 4 * lane);
          acc[i].x += x.x;
          acc[i].y += x.y;
          acc[i].z += x.z;
          acc[i].w += x.w;
        }
      }
    }
    auto finish = [&](int r, float m, float e, float l, float4 x) {
      const int rr = row0 + r;
      if (rr >= rows) return;
      // weights are at 2^(14 - E) * 2^s, the sum at 2^-m: the quotient's exponent
      const float f = m == -INFINITY ? 0.f : ex2(e - m - P_BIAS) / l;
      const int64_t tok = k.s.row0 + rr / a.G;
      const int head = k.h * a.G + rr % a.G;
      E y[4] = {from_float<E>(x.x * f), from_float<E>(x.y * f), from_float<E>(x.z * f), from_float<E>(x.w * f)};
      *reinterpret_cast<uint2*>(static_cast<E*>(a.out) + tok * a.o_tok + head * a.o_head + 4 * lane) =
          *reinterpret_cast<const uint2*>(y);
      if (a.lse != nullptr && lane == 0) a.lse[tok * a.Hq + head] = m + log2_acc(l);
    };
    if (k.t1 - k.t0 == k.blocks) {
#pragma unroll
      for (int i = 0; i < RPW; ++i)
        if (warp + i * C::WARPS < R) finish(warp + i * C::WARPS, rm[i], re[i], rl[i], acc[i]);
    } else {
      // Piece to the workspace: slot 2 cta (+ 1 for the task's first piece), so
      // that the two pieces a CTA may deliver do not meet.  The task's pieces lie
      // in CTAs c0 .. c1; its counter is that of c0, where only one task can
      // begin without ending.
      const long long k0 = u - k.t0, k1 = k0 + k.blocks;  // the task's units
      const int c0 = static_cast<int>(((k0 + 1) * parts - 1) / total), c1 = static_cast<int>((k1 * parts - 1) / total);
      constexpr int PART = R * (D + 4);
      float* part = a.parts + static_cast<size_t>(2 * blockIdx.x + (k.t0 == 0)) * PART;
#pragma unroll
      for (int i = 0; i < RPW; ++i) {
        const int r = warp + i * C::WARPS;
        if (r < R) {
          reinterpret_cast<float4*>(part + r * D)[lane] = acc[i];
          if (lane == 0) reinterpret_cast<float4*>(part + R * D)[r] = make_float4(rm[i], re[i], rl[i], 0.f);
        }
      }
      __threadfence();
      asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory");
      if (threadIdx.x == 0) {
        const unsigned int before = atom_add_acq_rel_gpu(a.counters + c0, 1u);
        const bool last = before == static_cast<unsigned int>(c1 - c0);
        if (last) a.counters[c0] = 0u;
        flags[1] = last;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory");
      if (flags[1]) {
        fence_acq_rel_gpu();
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
          const int r = warp + i * C::WARPS;
          if (r >= R) continue;
          float m = -INFINITY, e = -INFINITY, l = 0.f;
          for (int p = c0; p <= c1; ++p) {
            const float* q = a.parts + static_cast<size_t>(2 * p + (p == c0)) * PART;
            const float4 x = __ldcg(reinterpret_cast<const float4*>(q + R * D) + r);
            m = fmaxf(m, x.x);
            e = fmaxf(e, x.y);
          }
          const float mb = m == -INFINITY ? 0.f : m, eb = e == -INFINITY ? 0.f : e;
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p = c0; p <= c1; ++p) {
            const float* q = a.parts + static_cast<size_t>(2 * p + (p == c0)) * PART;
            const float4 x = __ldcg(reinterpret_cast<const float4*>(q + R * D) + r);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(q + r * D) + lane);
            l += x.z * ex2(x.x - mb);
            const float f = ex2(x.y - eb);
            s.x += y.x * f;
            s.y += y.y * f;
            s.z += y.z * f;
            s.w += y.w * f;
          }
          finish(r, m, e, l, s);
        }
      }
    }
    u += k.t1 - k.t0;
  }
}

constexpr int SMEM_MAX = 227 * 1024;

template <int NB, int NG>
int stage_count(int B) {
  using C = Cfg<NB, NG>;
  const int left = SMEM_MAX - C::FIXED - ((B + 1) * 4 + 127) / 128 * 128;
  const int n = left / HQ_KV8_PAGE_BYTES;
  return n < C::STAGE_MAX ? n : C::STAGE_MAX;
}

template <class E, int FMT, int NB, int NG>
hq_status launch(AttnArgs& a, int sms, cudaStream_t st) {
  using C = Cfg<NB, NG>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "kv8 attention setup");
  static DeviceOnce attrs;
  e = attrs.run(dev, [] {
    return cudaFuncSetAttribute(kv8_attn_kernel<E, FMT, NB, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
  });
  if (e != cudaSuccess) return cuda_fail(e, "kv8 attention setup");
  a.stages = stage_count<NB, NG>(a.c.B);
  a.groups = (a.G * a.max_new + C::R - 1) / C::R;
  const size_t smem = C::FIXED + ((a.c.B + 1) * 4 + 127) / 128 * 128 + static_cast<size_t>(a.stages) * HQ_KV8_PAGE_BYTES;
  kv8_attn_kernel<E, FMT, NB, NG><<<sms, C::THREADS, smem, st>>>(a);
  return cuda_status(cudaGetLastError(), "kv8 attention launch");
}

template <class E, int FMT>
hq_status launch_f(AttnArgs& a, int sms, cudaStream_t st) {
  if (a.G * static_cast<int64_t>(a.max_new) <= 8) return launch<E, FMT, 1, 2>(a, sms, st);
  return launch<E, FMT, 2, 2>(a, sms, st);
}

size_t counters_bytes(int sms) { return (static_cast<size_t>(sms) * 4 + 255) / 256 * 256; }

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

hq_status device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return cuda_status(e, "device query");
}

size_t attn_workspace(int rows, int sms) {
  const int R = rows <= 8 ? 8 : 16;
  return counters_bytes(sms) + static_cast<size_t>(2) * sms * R * (D + 4) * sizeof(float);
}

bool sizes_ok(const hq_kv8_cache* c, int Hq, int max_new) {
  return Hq > 0 && Hq % c->Hkv == 0 && max_new >= 0 && static_cast<int64_t>(Hq / c->Hkv) * max_new <= (1 << 24);
}

}  // namespace

hq_status kv8_validate(const hq_kv8_cache* c);

}  // namespace hq

extern "C" {

size_t hq_kv8_attn_workspace_bytes(const hq_kv8_cache* c, int32_t Hq, int32_t max_new) {
  if (hq::kv8_validate(c) != HQ_OK || !hq::sizes_ok(c, Hq, max_new)) return 0;
  int sms = 148;  // without a device: the B200's
  if (hq::device_sms(&sms) != HQ_OK) sms = 148;
  return hq::attn_workspace(Hq / c->Hkv * max_new, sms);
}

hq_status hq_kv8_attn(const hq_kv8_cache* c, int32_t dtype, const void* q, int64_t q_tok, int64_t q_head, int32_t Hq,
                      int32_t N, const int32_t* cu, const int32_t* kv_len, int32_t max_new, int32_t window, float sm_scale,
                      void* out, int64_t o_tok, int64_t o_head, float* lse, void* ws, size_t ws_bytes, hq_stream_t stream) {
  const hq_status st = hq::kv8_validate(c);
  if (st != HQ_OK) return st;
  if ((dtype != HQ_F16 && dtype != HQ_BF16) || N < 0 || window < 0 || !(sm_scale > 0.0f) || !hq::sizes_ok(c, Hq, max_new))
    return HQ_ERR_INVALID;
  if (!hq::aligned4(cu) || !hq::aligned4(kv_len) || (lse != nullptr && !hq::aligned4(lse))) return HQ_ERR_INVALID;
  if (N == 0 || max_new == 0) return HQ_OK;
  if (!hq::aligned16(q) || !hq::aligned16(out) || (q_tok | q_head | o_tok | o_head) % 8) return HQ_ERR_INVALID;
  // scratch is sized from the caller's max_new; fewer rows than that never need more
  int sms = 0;
  const hq_status ds = hq::device_sms(&sms);
  if (ds != HQ_OK) return ds;
  if (!hq::aligned16(ws) || ws_bytes < hq::attn_workspace(Hq / c->Hkv * max_new, sms)) return HQ_ERR_WORKSPACE;
  hq::AttnArgs a = {};
  a.c = *c;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.q_tok = q_tok;
  a.q_head = q_head;
  a.o_tok = o_tok;
  a.o_head = o_head;
  a.Hq = Hq;
  a.G = Hq / c->Hkv;
  a.N = N;
  a.max_new = max_new;
  a.window = window;
  a.cu = cu;
  a.kv_len = kv_len;
  a.scale = sm_scale * hq::LOG2E;
  a.counters = static_cast<unsigned int*>(ws);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + hq::counters_bytes(sms));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == HQ_F16)
    return c->fmt == HQ_KV8_E4M3 ? hq::launch_f<__half, HQ_KV8_E4M3>(a, sms, s) : hq::launch_f<__half, HQ_KV8_INT8>(a, sms, s);
  return c->fmt == HQ_KV8_E4M3 ? hq::launch_f<__nv_bfloat16, HQ_KV8_E4M3>(a, sms, s)
                               : hq::launch_f<__nv_bfloat16, HQ_KV8_INT8>(a, sms, s);
}

}  // extern "C"
