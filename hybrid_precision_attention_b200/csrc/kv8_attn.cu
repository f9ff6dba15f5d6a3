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
// depend on timing.  Within a CTA NG groups of 4 warps take every NG-th block of
// a task, 16 tokens a warp.  Each warp keeps a ring of its own 4 KB slices in
// flight by bulk copies (a slice is free again as soon as it is in registers, and
// no other warp is waited for) and its own running references, sums and
// accumulators.
//
// Two running references per row: m for the scores and, for the accumulators, E
// for score + log2(value scale), so that blocks whose scales lie far apart keep
// their precision.  A weight 2^(s - m) is summed in float32; its product with the
// value scale enters the matrix product as fp16 at 2^(s + log2 vscale - E + 6).
// The references are the exact maxima when they are set and stay as they are
// until a score passes m by 2^8 or a scale its reference by 2: the common block
// costs one comparison per score and one vote, and no cross-lane maximum.  The
// largest fp16 weight is then 2^15 and the smallest normal one 2^-20 of the
// reference.
#include <cuda_runtime.h>

#include <climits>
#include <type_traits>

#include "kv8.cuh"

namespace hq {
namespace {

constexpr float P_BIAS = 6.0f;     // log2 of the fp16 weight at both references
constexpr float P_SLACK = 8.0f;    // how far (log2) a score may pass m
constexpr float V_LIMIT = 128.0f;  // 2^(P_BIAS + 1): how far a value scale may pass its reference; 2^8 * 2^7 < 65504
constexpr int OS = D + 4;          // row stride (floats) of accumulators in shared memory: 4 rows of a store step 8 banks apart
constexpr int SLICE = 16 * D;      // bytes of one warp's 16 tokens of a page's K (or V) codes
constexpr int SLOT = 2 * SLICE + 16;  // K slice, V slice, scales

template <int NB>
struct Cfg {
  static constexpr int R = 8 * NB;              // rows of a task
  // 12 warps while a thread's accumulators and query operands (48 NB registers)
  // leave room in 168 registers, else 8 warps of up to 255
  static constexpr int NG = NB <= 2 ? 3 : 2;
  static constexpr int WARPS = 4 * NG;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int OBUF = WARPS * 8 * OS * 4;  // accumulators of 8 rows at a time
  static constexpr int RED = WARPS * R * 16;       // (m, E, l) of each warp's rows
  static constexpr int SLOTS = NB <= 2 ? 3 : 5;    // ring of a warp
  static constexpr int RING = WARPS * SLOTS * SLOT;
  static constexpr int FIXED = OBUF + RED + RING + WARPS * SLOTS * 8 + 128;
};

struct AttnArgs {
  hq_kv8_cache c;
  const void* q;
  void* out;
  float* lse;
  int64_t q_tok, q_head, o_tok, o_head;
  int Hq, G, N, max_new, window, groups;  // groups: tasks of a (sequence, kv head)
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

// Bounded wait on a slice of the ring; a copy that does not land within about a
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

template <class E, int FMT, int NB>
__global__ void __launch_bounds__(Cfg<NB>::THREADS, 1) kv8_attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<NB>;
  constexpr int R = C::R, NG = C::NG, SLOTS = C::SLOTS;
  extern __shared__ __align__(128) uint8_t sm[];
  float* obuf = reinterpret_cast<float*>(sm);                       // [warp][row of 8][OS]
  float4* red = reinterpret_cast<float4*>(sm + C::OBUF);            // [warp][row] (m, E, l, -)
  uint8_t* rings = sm + C::OBUF + C::RED;
  uint64_t* bars = reinterpret_cast<uint64_t*>(rings + C::RING);
  int* flags = reinterpret_cast<int*>(bars + C::WARPS * SLOTS);     // stop, last; 16.. warp totals of the plan
  int* prefix = reinterpret_cast<int*>(sm + C::FIXED);              // blocks (per task) of the sequences before b
  const int B = a.c.B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const hq_kv8_cache& c = a.c;

  // ---------------------------------------------------------------- plan
  uint64_t* full = bars + warp * SLOTS;
  if (lane == 0) {
    for (int i = 0; i < SLOTS; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) flags[0] = 0;
  int carry = 0;
  for (int b0 = 0; b0 < B; b0 += C::THREADS) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < B) {
      Kv8Seq s;
      kv8_seq(c, a.cu, a.kv_len, a.N, a.max_new, b, blockIdx.x == 0, s);
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
    if (lane == 31) flags[16 + warp] = x;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      const int y = flags[16 + w];
      if (w < warp) before += y;
      carry += y;
    }
    if (b < B) prefix[b] = before + x - n;
    __syncthreads();
  }
  const int per_seq = c.Hkv * a.groups;  // tasks of a sequence
  const long long total = static_cast<long long>(carry) * per_seq;
  const long long parts = min(total, static_cast<long long>(gridDim.x));  // CTAs with work: each has a block at least
  if (blockIdx.x >= parts) return;
  const long long u0 = total * blockIdx.x / parts, u1 = total * (blockIdx.x + 1) / parts;
  volatile int* stop = flags;

  // A task of the CTA's run: [t0, t1) of its blocks are ours.
  struct Task {
    int b, h, grp, begin, blocks, t0, t1;
    Kv8Seq s;
  };
  auto task_at = [&](long long u, Task& k) {
    const long long want = u / per_seq;  // the sequence holding unit u: prefix[b] <= want < prefix[b + 1]
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
    const int rel = static_cast<int>(u - static_cast<long long>(prefix[lo]) * per_seq);
    const int task = rel / k.blocks;
    k.h = task / a.groups;
    k.grp = task - k.h * a.groups;
    k.t0 = rel - task * k.blocks;
    k.t1 = static_cast<int>(min(static_cast<long long>(k.blocks), k.t0 + (u1 - u)));
  };

  const int g4 = warp >> 2, tt = warp & 3;  // group of 4 warps; the warp's 16 tokens of a block
  const int g = lane >> 2, t4 = lane & 3;

  // ------------------------------------------------------------ the warp's copies, SLOTS ahead
  // Blocks t = first, first + NG, .. of each task go to this group; the first
  // rotates with the task's number within the run.
  uint8_t* ring = rings + warp * SLOTS * SLOT;
  struct Cursor {
    long long u;              // units before the next task
    int t, end, b, ordinal;   // next block of the task (relative to its begin), end of the complete ones
    int batch, looked;        // pages of blocks batch, batch + NG, ..: lane i holds that of batch + i NG
    uint64_t page;
    size_t bh;
    int begin;
  } cur = {u0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
  auto first_of = [&](int t0, int ordinal) { return t0 + (g4 + ordinal) % NG; };
  auto issue = [&](int slot) {  // the next block's slice into the slot; false at the end of the run
    while (cur.t >= cur.end) {
      if (cur.u >= u1) return false;
      Task k;
      task_at(cur.u, k);
      cur.u += k.t1 - k.t0;
      cur.t = first_of(k.t0, cur.ordinal++);
      cur.end = min(k.t1, k.s.len / KV8_BLOCK - k.begin);  // the incomplete block is read where it lies
      cur.b = k.b;
      cur.bh = static_cast<size_t>(k.b) * c.Hkv + k.h;
      cur.begin = k.begin;
      cur.looked = 0;
    }
    if (cur.looked == 0 || cur.t >= cur.batch + 32 * NG) {
      cur.batch = cur.t;
      cur.looked = 1;
      const int t = cur.t + lane * NG;
      cur.page = t < cur.end ? reinterpret_cast<uint64_t>(kv8_page(c, cur.bh, cur.begin + t)) : 0;
    }
    const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, cur.page, (cur.t - cur.batch) / NG));
    cur.t += NG;
    if (lane == 0) {
      uint8_t* dst = ring + slot * SLOT;
      mbar_arrive_expect_tx(full + slot, SLOT);
      bulk_g2s(dst, page + tt * SLICE, SLICE, full + slot);
      bulk_g2s(dst + SLICE, page + HQ_KV8_V + tt * SLICE, SLICE, full + slot);
      bulk_g2s(dst + 2 * SLICE, page + HQ_KV8_KSCALE, 16, full + slot);
    }
    return true;
  };
  int issued = 0;
  while (issued < SLOTS && issue(issued)) ++issued;
  int slot = 0, phase = 0, taken = 0;
  bool ok = true;

  int ordinal = 0;
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
    int qp[NB][2];     // their positions (rows past the last: where they see all)
    float m_run[NB][2], e_run[NB][2], l_run[NB][2], ef[NB][2];  // ef = 2^(m - E + P_BIAS)
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
        // rows past the last have zero queries: their reference starts at their
        // score, 0, and no tile of theirs is ever masked or out of range
        qp[nb][i] = rr < rows ? k.s.first + rr / a.G : INT_MAX;
        m_run[nb][i] = rr < rows ? -INFINITY : 0.f;
        e_run[nb][i] = -INFINITY;
        l_run[nb][i] = ef[nb][i] = 0.f;
      }
    }
    // positions of the task's first and last real rows
    const int q_lo = k.s.first + row0 / a.G, q_hi = k.s.first + (min(row0 + R, rows) - 1) / a.G;

    float o[NB][8][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][mt][i] = 0.f;

    // one 16-token tile: kf, vf give the A operands of step s / output rows 16 mt
    // .. 16 mt + 15; ks, vs the scales of tokens g, g + 8 (vtop: the largest vs of
    // the tile); pos the first token's position
    auto tile = [&](auto masked, auto kf, auto vf, const float (&ks)[2], const float (&vs)[2], float vtop, int pos) {
      constexpr bool MASK = decltype(masked)::value;
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
          for (int i = 0; i < 4; ++i) sc[nb][i] = (sc[nb][i] + s2[nb][i]) * (qs[nb][i & 1] * ks[i >> 1]);
      }
      if (MASK) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // how far the token lies behind the query
            const int d = qp[nb][i & 1] - (pos + g + 8 * (i >> 1));
            if (d < 0 || (a.window > 0 && d >= a.window && qp[nb][i & 1] != INT_MAX)) sc[nb][i] = -INFINITY;
          }
      }
      bool far = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) far |= sc[nb][i] - m_run[nb][i & 1] > P_SLACK;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) far |= fmaxf(ef[nb][0], ef[nb][1]) * vtop > V_LIMIT;
      if (__any_sync(0xffffffffu, far)) {
        const float lv = log2f(vtop);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float ao[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mt = fmaxf(sc[nb][i], sc[nb][2 + i]);
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
            const float m_new = fmaxf(m_run[nb][i], mt), e_new = fmaxf(e_run[nb][i], mt + lv);
            const float mb = m_new == -INFINITY ? 0.f : m_new, eb = e_new == -INFINITY ? 0.f : e_new;
            l_run[nb][i] *= ex2(m_run[nb][i] - mb);
            ao[i] = ex2(e_run[nb][i] - eb);
            m_run[nb][i] = m_new;
            e_run[nb][i] = e_new;
            // bounded, so that a weight that underflowed stays 0 beside a far larger earlier score
            ef[nb][i] = e_new == -INFINITY ? 0.f : ex2(fminf(mb - eb + P_BIAS, 100.f));
          }
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nb][mt][i] *= ao[i & 1];
        }
      }
      uint32_t pf[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = ex2(sc[nb][i] - m_run[nb][i & 1]);
          if (MASK && sc[nb][i] == -INFINITY) p[i] = 0.f;  // also while m is -inf
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) l_run[nb][i] += p[i] + p[2 + i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] *= ef[nb][i & 1] * vs[i >> 1];
          if (MASK && sc[nb][i] == -INFINITY) p[i] = 0.f;  // a scale that is NaN stays behind the mask
        }
        pf[nb][0] = movmatrix_t(pack_f16x2(p[0], p[1]));
        pf[nb][1] = movmatrix_t(pack_f16x2(p[2], p[3]));
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        uint32_t f[4];
        vf(mt, f);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][mt], f[0], f[1], f[2], f[3], pf[nb][0], pf[nb][1]);
      }
    };

    for (int t = first_of(k.t0, ordinal); t < k.t1; t += NG) {
      const int p0 = (k.begin + t) * KV8_BLOCK, pos = p0 + tt * 16;
      if (p0 + KV8_BLOCK <= k.s.len) {
        ok = ok && ring_wait(full + slot, phase, c.err + k.b, stop);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* src = ring + slot * SLOT;
        uint4 kw[4], vw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kw[i] = reinterpret_cast<const uint4*>(src + i * 512)[lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) vw[i] = reinterpret_cast<const uint4*>(src + SLICE + i * 512)[lane];
        const float2 sc = *reinterpret_cast<const float2*>(src + 2 * SLICE);
        __syncwarp();  // every lane has its part: the slot takes the next slice
        ++taken;
        if (issue(slot)) ++issued;
        if (++slot == SLOTS) slot = 0, phase ^= 1;
        auto word = [](const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; };
        auto kf = [&](int s, uint32_t (&f)[4]) {
          // chunk (token half a, d half j) = 2 a + j; word s % 4 of it
          kv8_half4<FMT>(word(kw[s >> 2], s & 3), f[0], f[2]);
          kv8_half4<FMT>(word(kw[2 + (s >> 2)], s & 3), f[1], f[3]);
        };
        auto vf = [&](int mt, uint32_t (&f)[4]) {
          kv8_half4<FMT>(word(vw[mt >> 1], (mt & 1) * 2), f[0], f[2]);
          kv8_half4<FMT>(word(vw[mt >> 1], (mt & 1) * 2 + 1), f[1], f[3]);
        };
        const float ks[2] = {sc.x, sc.x}, vs[2] = {sc.y, sc.y};
        // seen whole by every row?
        if (pos + 15 <= q_lo && (a.window <= 0 || pos > q_hi - a.window))
          tile(std::false_type{}, kf, vf, ks, vs, sc.y, pos);
        else
          tile(std::true_type{}, kf, vf, ks, vs, sc.y, pos);
      } else if (pos < k.s.len) {
        // the incomplete block, in 16 bits: rows past the length hold finite
        // values of earlier blocks or zeros and are masked
        const int half = (k.begin + t) & 1;
        const uint4* tk = reinterpret_cast<const uint4*>(c.tail_k + (bh * 2 + half) * KV8_BLOCK * D + tt * 2048);
        const uint4* tv = reinterpret_cast<const uint4*>(c.tail_v + (bh * 2 + half) * KV8_BLOCK * D + tt * 2048);
        const float* ts = c.tail_scale + bh * 2 * HQ_KV8_TAIL + half * KV8_BLOCK + tt * 16 + g;
        const bool in0 = pos + g < k.s.len, in1 = pos + g + 8 < k.s.len;
        const float ks[2] = {in0 ? ts[0] : 1.f, in1 ? ts[8] : 1.f};
        const float vs[2] = {in0 ? ts[HQ_KV8_TAIL] : 0.f, in1 ? ts[HQ_KV8_TAIL + 8] : 0.f};
        float vtop = fmaxf(vs[0], vs[1]);  // ignores NaN
        vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, 4));
        vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, 8));
        vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, 16));
        if (!(vtop > 0.f)) vtop = 1.f;
        uint32_t kw[4][8], vw[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *reinterpret_cast<uint4*>(&kw[i][0]) = tk[(i * 32 + lane) * 2];
          *reinterpret_cast<uint4*>(&kw[i][4]) = tk[(i * 32 + lane) * 2 + 1];
        }
        auto kf = [&](int s, uint32_t (&f)[4]) {
          f[0] = kw[s >> 2][(s & 3) * 2];
          f[2] = kw[s >> 2][(s & 3) * 2 + 1];
          f[1] = kw[2 + (s >> 2)][(s & 3) * 2];
          f[3] = kw[2 + (s >> 2)][(s & 3) * 2 + 1];
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *reinterpret_cast<uint4*>(&vw[i][0]) = tv[(i * 32 + lane) * 2];
          *reinterpret_cast<uint4*>(&vw[i][4]) = tv[(i * 32 + lane) * 2 + 1];
        }
        auto vf = [&](int mt, uint32_t (&f)[4]) {
          const int w = (mt & 1) * 4;
          f[0] = vw[mt >> 1][w];
          f[2] = vw[mt >> 1][w + 1];
          f[1] = vw[mt >> 1][w + 2];
          f[3] = vw[mt >> 1][w + 3];
        };
        tile(std::true_type{}, kf, vf, ks, vs, vtop, pos);
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
    const bool whole = k.t1 - k.t0 == k.blocks;
    // Pieces of a task that CTAs share lie in the workspace, slot 2 cta (+ 1 for
    // the task's first piece): the two pieces a CTA may deliver do not meet.  The
    // task's pieces come from CTAs c0 .. c1 and are counted by c0's counter: one
    // task at most begins in a CTA without ending there.
    constexpr int PART = R * (D + 4);
    float* part = a.parts + static_cast<size_t>(2 * blockIdx.x + (k.t0 == 0)) * PART;
    auto finish = [&](int r, float m, float e, float l, float4 x) {
      const int rr = row0 + r;
      if (rr >= rows) return;
      // accumulators are at 2^(P_BIAS - E), the sum at 2^-m: the quotient's exponent
      const float f = m == -INFINITY ? 0.f : ex2(e - m - P_BIAS) / l;
      const int64_t tok = k.s.row0 + rr / a.G;
      const int head = k.h * a.G + rr % a.G;
      E y[4] = {from_float<E>(x.x * f), from_float<E>(x.y * f), from_float<E>(x.z * f), from_float<E>(x.w * f)};
      *reinterpret_cast<uint2*>(static_cast<E*>(a.out) + tok * a.o_tok + head * a.o_head + 4 * lane) =
          *reinterpret_cast<const uint2*>(y);
      if (a.lse != nullptr && lane == 0) a.lse[tok * a.Hq + head] = m + log2f(l);
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      __syncthreads();  // red is there; the buffer's earlier readers are done
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * t4 + i;
        float e = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) e = fmaxf(e, red[w * R + 8 * nb + r].y);
        const float f = e == -INFINITY ? 1.f : ex2(e_run[nb][i] - e);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          obuf[(warp * 8 + r) * OS + mt * 16 + g] = o[nb][mt][i] * f;
          obuf[(warp * 8 + r) * OS + mt * 16 + g + 8] = o[nb][mt][2 + i] * f;
        }
      }
      // row 8 nb + warp of the first 8 warps: elements 4 lane .. 4 lane + 3
      float m = -INFINITY, e = -INFINITY, l = 0.f;
      if (warp < 8) {
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float4 x = red[w * R + 8 * nb + warp];
          m = fmaxf(m, x.x);
          e = fmaxf(e, x.y);
        }
        const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float4 x = red[w * R + 8 * nb + warp];
          l += x.z * ex2(x.x - mb);
        }
      }
      __syncthreads();
      if (warp < 8) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(obuf + (w * 8 + warp) * OS + 4 * lane);
          s.x += x.x;
          s.y += x.y;
          s.z += x.z;
          s.w += x.w;
        }
        const int r = 8 * nb + warp;
        if (whole) {
          finish(r, m, e, l, s);
        } else {
          reinterpret_cast<float4*>(part + r * D)[lane] = s;
          if (lane == 0) reinterpret_cast<float4*>(part + R * D)[r] = make_float4(m, e, l, 0.f);
        }
      }
    }
    if (!whole) {
      const long long k0 = u - k.t0, k1 = k0 + k.blocks;  // the task's units
      const int c0 = static_cast<int>(((k0 + 1) * parts - 1) / total), c1 = static_cast<int>((k1 * parts - 1) / total);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const unsigned int before = atom_add_acq_rel_gpu(a.counters + c0, 1u);
        const bool last = before == static_cast<unsigned int>(c1 - c0);
        if (last) a.counters[c0] = 0u;
        flags[1] = last;
      }
      __syncthreads();
      if (flags[1]) {
        fence_acq_rel_gpu();
        for (int r = warp; r < R; r += C::WARPS) {
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
    ++ordinal;
    u += k.t1 - k.t0;
  }
  // copies that were not waited for (after a wait that gave up) land before the
  // CTA gives its shared memory back
  if (!ok && lane == 0) {
    int never = 0;
    for (; taken < issued; ++taken) ring_wait(full + taken % SLOTS, (taken / SLOTS) & 1, c.err, &never);
  }
}

constexpr int SMEM_MAX = 227 * 1024;

template <class E, int FMT, int NB>
hq_status launch(AttnArgs& a, int sms, cudaStream_t st) {
  using C = Cfg<NB>;
  static_assert(C::FIXED + (HQ_KV8_MAX_BATCH + 1) * 4 <= SMEM_MAX, "shared memory of the largest batch");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "kv8 attention setup");
  static DeviceOnce attrs;
  e = attrs.run(dev, [] {
    return cudaFuncSetAttribute(kv8_attn_kernel<E, FMT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
  });
  if (e != cudaSuccess) return cuda_fail(e, "kv8 attention setup");
  a.groups = (a.G * a.max_new + C::R - 1) / C::R;
  kv8_attn_kernel<E, FMT, NB><<<sms, C::THREADS, C::FIXED + (a.c.B + 1) * 4, st>>>(a);
  return cuda_status(cudaGetLastError(), "kv8 attention launch");
}

// Rows of a task, in eights: as many as there are, up to 4; beyond that tasks of 32 rows.
int row_eights(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4; }

template <class E, int FMT>
hq_status launch_f(AttnArgs& a, int sms, cudaStream_t st) {
  switch (row_eights(a.G * a.max_new)) {
    case 1: return launch<E, FMT, 1>(a, sms, st);
    case 2: return launch<E, FMT, 2>(a, sms, st);
    case 3: return launch<E, FMT, 3>(a, sms, st);
    default: return launch<E, FMT, 4>(a, sms, st);
  }
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
  const int R = 8 * row_eights(rows);
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
