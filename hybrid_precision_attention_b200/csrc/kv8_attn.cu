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
// Work: the tasks (sequence, kv head, 8 NB rows of it) have their blocks laid end to
// end and cut into gridDim runs, equal to a block.  A task that one CTA holds
// whole is finished there; the pieces of the others go to the workspace and the
// CTA that delivers a task's last piece joins them in order, so that results do
// not depend on timing.  Short tasks are not cut.  Within a CTA NG groups of warps
// take every NG-th block of a task, 32 tokens a warp.  Each warp keeps a ring of
// its own slices of the pages in flight by bulk copies (no other warp is waited
// for) and its own running references, sums and accumulators.  Registers are what
// bounds the tokens of a step and the warps: the query operands stand in shared memory
// and values stay in the slot until they are needed (with both in registers 24
// rows left room for 16 tokens a step: 64 sequences of 1K to 8K 183 us, now 131 us).
//
// Two running references per row: m for the scores and, for the accumulators, E
// for score + log2(value scale), so that blocks whose scales lie far apart keep
// their precision.  A weight 2^(s - m) is summed in float32; its product with the
// value scale enters the matrix product as fp16 at 2^(s + log2 vscale - E + 6): the type
// in which codes are exact and a product with them is one instruction.  That rounding adds a
// quarter to a third to the error of fp16 outputs (2.6e-4 to 2.9e-4 of their size, their own
// rounding is 2.1e-4).
// The references are the exact maxima when they are set and stay as they are
// until a score passes m by 2^8 or a weight E by 2^9: the common block
// costs one comparison per score and one vote, and no cross-lane maximum.  The
// largest fp16 weight is then 2^15 and the smallest normal one 2^-20 of the
// reference.  (A bound on the weights by m in place of the weights themselves had E
// set anew on page after page where the largest score belonged to a small value: 24 rows
// 143 us against 135.)
//
// Measured (8 kv heads): 64 sequences of 1K to 16K, a token each, 8 rows: 183 us, 6.3 TB/s of
// codes, the copy rate; 64 of 1K to 8K: 8 rows 98 us, 6.0 TB/s, 16 rows 106 us, 24 rows 135 us,
// 4.4 TB/s; 16 windows of 4096, 20 rows: 45 us, 3.0 TB/s, bound by the latencies of a
// step (two warps a scheduler) and by the tasks' ends.  24 rows take 255 registers and spill 290
// to 360 bytes a thread; where in the code is not known.  One sequence of 32K: 18.8 us,
// 3.6 TB/s: 10.4 us of it are the pages at the copy rate, the others launch, plan, first copies
// and the join of 19 pieces.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "kv8.cuh"

namespace hq {
size_t kv8_attn_tc_parts(int64_t rows, int sms);
hq_status launch_kv8_attn_tc(const Kv8AttnArgs& a, int dtype, int sms, cudaStream_t st);

namespace {

constexpr float P_BIAS = 6.0f;     // log2 of the fp16 weight at both references
constexpr float P_SLACK = 8.0f;    // how far (log2) a score may pass m
constexpr float W_TOP = 15.0f;     // log2 of the largest fp16 weight
// log2 of the largest factor of weights, 2^(m - E + P_BIAS): E stays above m + P_BIAS - P_TOP, so that the factor and
// the inverse that undoes it at the end are both normal numbers (value scales below 2^(P_BIAS - P_TOP) then give
// smaller weights), and a weight that underflowed stays 0 beside a far larger earlier score
constexpr float P_TOP = 120.0f;
constexpr int TASK_UNITS = 12;     // what a task costs besides its blocks, in blocks (about 6000 cycles of 500 each)
constexpr int OS = D + 4;          // row stride (floats) of accumulators in shared memory: 4 rows of a store step 8 banks apart

template <int NB, int W>
struct Cfg {
  static constexpr int R = 8 * NB;            // rows of a task
  static constexpr int MT = 2;                // 16-token tiles of a page that a warp takes in one step
  static constexpr int WARPS = W;             // of up to 255 registers
  static constexpr int CTAS = 8 / W;          // on an SM
  static constexpr int THREADS = WARPS * 32;
  static constexpr int PW = 4 / MT;           // warps of a group, which share a page
  static constexpr int NG = WARPS / PW;       // groups
  static constexpr int SLICE = MT * 16 * D;   // bytes of a warp's part of a page's K (or V) codes
  static constexpr int SLOT = 2 * SLICE + 16; // K slice, V slice, scales
  static constexpr int SLOTS = 2;             // ring of a warp
  static constexpr int OW = W < 4 ? W : 4;    // warps whose accumulators are in shared memory at a time
  static constexpr int OBUF = OW * 8 * OS * 4;     // of 8 rows
  static constexpr int RED = WARPS * R * 16;       // (m, E, l) of each warp's rows
  static constexpr int Q = NB * 2048 + R * 4;      // query operands [NB][4][lane] of 16 bytes; multipliers of rows
  static constexpr int RING = WARPS * SLOTS * SLOT;
  static constexpr int AHEAD = 80;                 // a warp's copy cursor
  static constexpr int FIXED = OBUF + RED + Q + RING + WARPS * (SLOTS * 8 + AHEAD) + 32 * 8 + 16;
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

template <class E, int FMT, int NB, int W>
__global__ void __launch_bounds__(Cfg<NB, W>::THREADS, Cfg<NB, W>::CTAS) kv8_attn_kernel(const __grid_constant__ Kv8AttnArgs a) {
  using C = Cfg<NB, W>;
  constexpr int R = C::R, NG = C::NG, SLOTS = C::SLOTS, MT = C::MT, SLICE = C::SLICE, SLOT = C::SLOT;
  extern __shared__ __align__(128) uint8_t sm[];
  float* obuf = reinterpret_cast<float*>(sm);                       // [warp][row of 8][OS]
  float4* red = reinterpret_cast<float4*>(sm + C::OBUF);            // [warp][row] (m, E, l, -)
  uint4* q_sh = reinterpret_cast<uint4*>(sm + C::OBUF + C::RED);
  float* q_mul = reinterpret_cast<float*>(q_sh + NB * 128);
  uint8_t* rings = sm + C::OBUF + C::RED + C::Q;
  uint64_t* bars = reinterpret_cast<uint64_t*>(rings + C::RING);
  uint64_t* sums = bars + C::WARPS * SLOTS;                         // the plan's sums and maxima of each warp
  uint8_t* ahead = reinterpret_cast<uint8_t*>(sums + 32);
  int* flags = reinterpret_cast<int*>(ahead + C::WARPS * C::AHEAD);  // stop, last
  uint64_t* prefix = reinterpret_cast<uint64_t*>(sm + C::FIXED);
  const int B = a.c.B;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const hq_kv8_cache& c = a.c;

  // ---------------------------------------------------------------- plan
  uint64_t* full = bars + warp * SLOTS;
  if (lane == 0) {
    for (int i = 0; i < SLOTS; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 2) flags[threadIdx.x] = 0;
  chained();
  auto groups_of = [&](const Kv8Seq& s) { return (s.n * a.G + R - 1) / R; };  // of rows
  // prefix[b]: units (of one kv head) of the sequences before b, in the low half,
  // and their tasks in the high half
  uint64_t carry = 0;
  int longest = 0;
  for (int b0 = 0; b0 < B; b0 += C::THREADS) {
    const int b = b0 + threadIdx.x;
    int n = 0, groups = 0;
    if (b < B) {
      Kv8Seq s;
      kv8_seq(c, a.cu, a.kv_len, a.N, a.max_new, b, blockIdx.x == 0, s);
      int begin, end;
      seq_blocks(s, a.window, begin, end);
      n = end - begin;
      groups = groups_of(s);
    }
    const uint64_t mine = n > 0 ? static_cast<uint64_t>(groups) << 32 | static_cast<uint32_t>(groups * (n + TASK_UNITS)) : 0ull;
    uint64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int top = __reduce_max_sync(0xffffffffu, n);
    if (lane == 31) {
      sums[warp] = x;
      sums[16 + warp] = top;
    }
    __syncthreads();
    uint64_t before = carry;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      const uint64_t y = sums[w];
      if (w < warp) before += y;
      carry += y;
      longest = max(longest, static_cast<int>(sums[16 + w]));
    }
    if (b < B) prefix[b] = before + x - mine;
    __syncthreads();
  }
  // The units that are dealt out: a task is its blocks and TASK_UNITS more for
  // what it costs besides them; or, where every task is short and none need share
  // a CTA with another, one unit, so that no task is cut (its pieces' way through
  // the workspace takes longer than 24 blocks).
  const uint32_t per_seq = c.Hkv;  // what the prefixes count comes once for each kv head
  const uint32_t tasks = static_cast<uint32_t>(carry >> 32) * per_seq;
  const bool uncut = longest <= 24 && tasks <= gridDim.x;
  const uint32_t total = uncut ? tasks : static_cast<uint32_t>(carry) * per_seq;
  const uint32_t parts = min(total, gridDim.x);  // CTAs with work: a unit each at least
  if (blockIdx.x >= parts) return;
  // the first `more` runs have a unit more than the others
  const uint32_t run = total / parts, more = total - run * parts;
  const uint32_t u0 = run * blockIdx.x + min(blockIdx.x, more), u1 = u0 + run + (blockIdx.x < more);
  auto cta_of = [&](uint32_t u) { return u < more * (run + 1) ? u / (run + 1) : more + (u - more * (run + 1)) / run; };
  auto before_of = [&](int b) { return uncut ? static_cast<uint32_t>(prefix[b] >> 32) : static_cast<uint32_t>(prefix[b]); };
  volatile int* stop = flags;

  // A task of the CTA's run: [t0, t1) of its blocks are ours (none where the run
  // begins behind them), `units` of the run.
  struct Task {
    int b, h, row0, begin, blocks, t0, t1;  // rows row0 .. row0 + R - 1 of the kv head
    uint32_t units;
    Kv8Seq s;
  };
  auto seq_of = [&](Task& k) {
    kv8_seq(c, a.cu, a.kv_len, a.N, a.max_new, k.b, false, k.s);
    int end;
    seq_blocks(k.s, a.window, k.begin, end);
    k.blocks = end - k.begin;
  };
  auto span_of = [&](uint32_t u, Task& k) {
    k.units = uncut ? 1u : min(static_cast<uint32_t>(k.blocks + TASK_UNITS - k.t0), u1 - u);
    k.t1 = uncut ? k.blocks : min(k.blocks, k.t0 + static_cast<int>(k.units));
  };
  auto task_at = [&](uint32_t u, Task& k) {  // the task that holds unit u
    const uint32_t want = u / per_seq;       // in the sequence with before_of(b) <= want < before_of(b + 1)
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before_of(mid) <= want) lo = mid; else hi = mid;
    }
    k.b = lo;
    seq_of(k);
    const uint32_t rel = u - before_of(lo) * per_seq;
    const uint32_t each = uncut ? 1u : k.blocks + TASK_UNITS, task = rel / each;
    const int groups = groups_of(k.s);
    k.h = task / groups;
    k.row0 = (task - k.h * groups) * R;
    k.t0 = rel - task * each;
    span_of(u, k);
  };
  auto next_task = [&](uint32_t u, Task& k) {  // the task after k, which begins with unit u < u1
    k.t0 = 0;
    if ((k.row0 += R) >= k.s.n * a.G) {
      k.row0 = 0;
      if (++k.h == c.Hkv) {
        k.h = 0;
        do {
          ++k.b;
          seq_of(k);
        } while (k.blocks == 0);
      }
    }
    span_of(u, k);
  };

  const int g4 = warp / C::PW, tt = warp % C::PW;  // group; the warp's 16 MT tokens of a block
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t u_first = u0;
  Task k;
  task_at(u0, k);
  if (k.t0 >= k.blocks) {  // the run begins behind a task's blocks
    u_first += k.units;
    if (u_first >= u1) return;
    next_task(u_first, k);
  }

  // raw query rows 8 nb + g of a task's (elements 16 t4 .. and 64 + 16 t4 ..)
  auto load_q = [&](const Task& k, int nb, uint4 (&v)[4]) {
    const int r = k.row0 + 8 * nb + g;
    if (r < k.s.n * a.G) {
      const E* p = static_cast<const E*>(a.q) + static_cast<int64_t>(k.s.row0 + r / a.G) * a.q_tok +
                   static_cast<int64_t>(k.h * a.G + r % a.G) * a.q_head + 16 * t4;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[2 * j] = *reinterpret_cast<const uint4*>(p + 64 * j);
        v[2 * j + 1] = *reinterpret_cast<const uint4*>(p + 64 * j + 8);
      }
    } else {
      v[0] = v[1] = v[2] = v[3] = make_uint4(0u, 0u, 0u, 0u);
    }
  };

  // ------------------------------------------------------------ the warp's copies, SLOTS ahead
  // Blocks t = first, first + NG, .. of each task go to this group; the first
  // rotates with the task's number within the run.
  uint8_t* ring = rings + warp * SLOTS * SLOT;
  // The pool pages of the warp's blocks are looked up 32 at a time, lane i the
  // i-th, and a lookup ahead of their use.  The cursor lies in shared memory: the
  // warp's registers are full.  Every lane reads the same words.
  struct Ahead {
    Task k;
    uint32_t u;           // first unit of its task
    int ordinal, t;       // the task's number in the run, the next block to look up
  };
  static_assert(sizeof(Ahead) <= C::AHEAD, "the cursor's place");
  Ahead& ah = *reinterpret_cast<Ahead*>(ahead + warp * C::AHEAD);
  // a task's queries are fetched while the one before it is joined, the first's here
  uint4 qv[4];
  if (warp < NB) load_q(k, warp, qv);
  auto first_of = [&](int t0, int ordinal) { return t0 + (g4 + ordinal) % NG; };
  struct Pages {
    int n, at, b;         // how many (0: the run has no more), the next one, their sequence
    int idx;              // the lane's page, -1: outside the pool
  } now, then;
  auto look_up = [&](Pages& x) {
    while (true) {
      const int left = min(ah.k.t1, ah.k.s.len / KV8_BLOCK - ah.k.begin) - ah.t;  // the incomplete block is read where it lies
      if (left > 0) {
        x.n = min(32, (left + NG - 1) / NG);
        x.at = 0;
        x.b = ah.k.b;
        if (lane < x.n)
          x.idx = static_cast<int>(kv8_page_index(c, static_cast<size_t>(ah.k.b) * c.Hkv + ah.k.h, ah.k.begin + ah.t + lane * NG));
        __syncwarp();
        if (lane == 0) ah.t += 32 * NG;
        __syncwarp();
        return;
      }
      x.n = x.at = 0;
      const uint32_t u = ah.u + ah.k.units;
      if (u >= u1) return;
      Task n = ah.k;
      next_task(u, n);
      const int ordinal = ah.ordinal + 1;
      __syncwarp();
      if (lane == 0) ah = Ahead{n, u, ordinal, first_of(n.t0, ordinal)};
      __syncwarp();
    }
  };
  if (lane == 0) ah = Ahead{k, u_first, 0, first_of(k.t0, 0)};
  __syncwarp();
  now = Pages{0, 0, 0, 0};
  look_up(then);
  auto issue = [&](int slot) {  // the next block's slice into the slot; false at the end of the run
    if (now.at == now.n) {
      if (then.n == 0) return false;
      now = then;
      look_up(then);
    }
    int idx = __shfl_sync(0xffffffffu, now.idx, now.at);
    ++now.at;
    if (idx < 0) {
      if (lane == 0) kv8_err(c, now.b, HQ_DEVERR_PAGE);
      idx = 0;
    }
    const uint8_t* page = c.pages + static_cast<size_t>(idx) * HQ_KV8_PAGE_BYTES;
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

  // query rows as B operands: lane (g, t4) holds row g (+ 8 nb), elements
  // 64 j + 16 t4 + 4 u + {0..3} at step 4 j + u, the elements that the K codes'
  // 16-byte chunk t4 of half j gives at that step.  Returns the row's multiplier.
  auto operands = [&](const uint4 (&v)[4], uint32_t (&f)[16]) {
    float mul = 1.0f;
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
      for (int i = 0; i < 16; ++i) f[i] = pack_f16x2(to_float(e[2 * i]) * inv, to_float(e[2 * i + 1]) * inv);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = reinterpret_cast<const uint32_t*>(v)[i];
    }
    return mul;
  };
  // the fetched queries into shared memory, 8 rows a warp; a barrier follows
  auto stage_q = [&]() {
    if (warp < NB) {
      uint32_t f[16];
      const float mul = operands(qv, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) q_sh[(warp * 4 + i) * 32 + lane] = make_uint4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      if (t4 == 0) q_mul[8 * warp + g] = mul * a.scale;
    }
  };
  stage_q();
  __syncthreads();

  int ordinal = 0;
  for (uint32_t u = u_first;;) {
    const size_t bh = static_cast<size_t>(k.b) * c.Hkv + k.h;
    const int rows = k.s.n * a.G;

    float qs[NB][2];   // multiplier of the scores of rows 2 t4, 2 t4 + 1
    int qp[NB][2];     // their positions (rows past the last: where they see all)
    float m_run[NB][2], e_run[NB][2], l_run[NB][2], ef[NB][2];  // ef = 2^(m - E + P_BIAS)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qs[nb][i] = q_mul[8 * nb + 2 * t4 + i];
        const int rr = k.row0 + 8 * nb + 2 * t4 + i;
        // rows past the last have zero queries: their reference starts at their
        // score, 0, and no tile of theirs is ever masked or out of range
        qp[nb][i] = rr < rows ? k.s.first + rr / a.G : INT_MAX;
        m_run[nb][i] = rr < rows ? -INFINITY : 0.f;
        e_run[nb][i] = -INFINITY;
        l_run[nb][i] = ef[nb][i] = 0.f;
      }
    }
    // positions of the task's first and last real rows
    const int q_lo = k.s.first + k.row0 / a.G, q_hi = k.s.first + (min(k.row0 + R, rows) - 1) / a.G;

    float o[NB][8][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][mt][i] = 0.f;

    // NT 16-token tiles: kf, vf give the A operands of step s / output rows 16 d
    // .. 16 d + 15 of tile j; ks, vs the scales of its tokens g, g + 8 (`own`: of each token its
    // own, else the same of all); pos the first token's position
    auto tiles = [&](auto count, auto masked, auto own, auto kf, auto vf, const float (&ks)[2], const float (&vs)[2], int pos) {
      constexpr int NT = decltype(count)::value;
      constexpr bool MASK = decltype(masked)::value, OWN = decltype(own)::value;
      float sc[NT][NB][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[j][nb][i] = 0.f;
      uint4 qw[NB];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s % 2 == 0) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) qw[nb] = q_sh[(nb * 4 + s / 2) * 32 + lane];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t f[4];
          kf(j, s, f);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma16816(sc[j][nb], f[0], f[1], f[2], f[3], s & 1 ? qw[nb].z : qw[nb].x, s & 1 ? qw[nb].w : qw[nb].y);
        }
      }
      bool far = OWN;  // the first of the task's
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // how far a score may pass m: by P_SLACK, and no further than its weight stays below 2^W_TOP
        float most[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) most[i] = OWN ? P_SLACK : fminf(P_SLACK, W_TOP - lg2_approx(ef[nb][i] * vs[0]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mul = qs[nb][i & 1] * ks[i >> 1];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            sc[j][nb][i] *= mul;
            if (MASK) {
              // how far the token lies behind the query
              const int d = qp[nb][i & 1] - (pos + 16 * j + g + 8 * (i >> 1));
              if (d < 0 || (a.window > 0 && d >= a.window && qp[nb][i & 1] != INT_MAX)) sc[j][nb][i] = -INFINITY;
            }
            far |= sc[j][nb][i] - m_run[nb][i & 1] > most[i & 1];
          }
        }
      }
      if (__any_sync(0xffffffffu, far)) {
        const float lv[2] = {log2f(vs[0]), log2f(vs[1])};
        const float low = (OWN ? 0.f : fmaxf(lv[0], 0.f)) + (P_BIAS - P_TOP);  // the factor times the scale is finite, too
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float ao[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mt = -INFINITY;
#pragma unroll
            for (int j = 0; j < NT; ++j) mt = fmaxf(mt, fmaxf(sc[j][nb][i], sc[j][nb][2 + i]));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
            float et = mt + lv[0];  // the largest score + log2(value scale) of what the row sees; NaN is passed over
            if (OWN) {
              et = -INFINITY;
#pragma unroll
              for (int j = 0; j < NT; ++j) et = fmaxf(et, fmaxf(sc[j][nb][i] + lv[0], sc[j][nb][2 + i] + lv[1]));
              et = fmaxf(et, __shfl_xor_sync(0xffffffffu, et, 4));
              et = fmaxf(et, __shfl_xor_sync(0xffffffffu, et, 8));
              et = fmaxf(et, __shfl_xor_sync(0xffffffffu, et, 16));
            }
            const float m_new = fmaxf(m_run[nb][i], mt), e_new = fmaxf(fmaxf(e_run[nb][i], et), m_new + low);
            const float mb = m_new == -INFINITY ? 0.f : m_new, eb = e_new == -INFINITY ? 0.f : e_new;
            l_run[nb][i] *= ex2(m_run[nb][i] - mb);
            ao[i] = ex2(e_run[nb][i] - eb);
            m_run[nb][i] = m_new;
            e_run[nb][i] = e_new;
            ef[nb][i] = e_new == -INFINITY ? 0.f : ex2(mb - eb + P_BIAS);
          }
#pragma unroll
          for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nb][d][i] *= ao[i & 1];
        }
      }
      uint32_t pf[NT][NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = OWN ? vs[i >> 1] : ef[nb][i & 1] * vs[i >> 1];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = ex2(sc[j][nb][i] - m_run[nb][i & 1]);
            if (MASK && sc[j][nb][i] == -INFINITY) p[i] = 0.f;  // also while m is -inf
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) l_run[nb][i] += p[i] + p[2 + i];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = (OWN ? p[i] * ef[nb][i & 1] : p[i]) * w[i];
            if (MASK && sc[j][nb][i] == -INFINITY) p[i] = 0.f;  // a scale that is NaN stays behind the mask
          }
          pf[j][nb][0] = movmatrix_t(pack_f16x2(p[0], p[1]));
          pf[j][nb][1] = movmatrix_t(pack_f16x2(p[2], p[3]));
        }
      }
#pragma unroll
      for (int d = 0; d < 8; ++d)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t f[4];
          vf(j, d, f);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][d], f[0], f[1], f[2], f[3], pf[j][nb][0], pf[j][nb][1]);
        }
    };

    // The incomplete block first, in 16 bits from where it lies, a tile to each of
    // four warps: rows past the length hold finite values of earlier blocks or
    // zeros and are masked.
    const int full_end = min(k.t1, k.s.len / KV8_BLOCK - k.begin);
    if (full_end < k.t1 && warp % (C::WARPS / 4) == 0) {
      const int t16 = warp / (C::WARPS / 4), blk = k.begin + full_end, pos = blk * KV8_BLOCK + t16 * 16;
      if (pos < k.s.len) {
        const size_t half = bh * 2 + (blk & 1);
        const uint4* tk = reinterpret_cast<const uint4*>(c.tail_k + half * KV8_BLOCK * D + t16 * 2048);
        const uint4* tv = reinterpret_cast<const uint4*>(c.tail_v + half * KV8_BLOCK * D + t16 * 2048);
        const float* ts = c.tail_scale + bh * 2 * HQ_KV8_TAIL + (blk & 1) * KV8_BLOCK + t16 * 16 + g;
        uint32_t kw[4][8], vw[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *reinterpret_cast<uint4*>(&kw[i][0]) = tk[(i * 32 + lane) * 2];
          *reinterpret_cast<uint4*>(&kw[i][4]) = tk[(i * 32 + lane) * 2 + 1];
        }
        const bool in0 = pos + g < k.s.len, in1 = pos + g + 8 < k.s.len;
        const float ks[2] = {in0 ? ts[0] : 1.f, in1 ? ts[8] : 1.f};
        float vs[2] = {in0 ? ts[HQ_KV8_TAIL] : 0.f, in1 ? ts[HQ_KV8_TAIL + 8] : 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *reinterpret_cast<uint4*>(&vw[i][0]) = tv[(i * 32 + lane) * 2];
          *reinterpret_cast<uint4*>(&vw[i][4]) = tv[(i * 32 + lane) * 2 + 1];
        }
        // the largest magnitudes of tokens 2 t4, 2 t4 + 1 (even words) and of those 8 behind (odd words)
        uint32_t top[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 32; ++i) top[i & 1] = kv8_top2(top[i & 1], vw[i / 8][i % 8]);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
          for (int o = 4; o < 32; o *= 2) top[z] = kv8_top2(top[z], __shfl_xor_sync(0xffffffffu, top[z], o));
          const TailUp up(top[z]);
#pragma unroll
          for (int i = 0; i < 16; ++i) vw[i / 4][i % 4 * 2 + z] = up(vw[i / 4][i % 4 * 2 + z]);
          // of token g (+ 8): with the lanes whose t4 is g / 2
          vs[z] = kv8_tail_vscale(vs[z], __shfl_sync(0xffffffffu, top[z], g >> 1) >> (g & 1) * 16 & 0x7fffu);
        }
        auto kf = [&](int, int s, uint32_t (&f)[4]) {
          f[0] = kw[s >> 2][(s & 3) * 2];
          f[2] = kw[s >> 2][(s & 3) * 2 + 1];
          f[1] = kw[2 + (s >> 2)][(s & 3) * 2];
          f[3] = kw[2 + (s >> 2)][(s & 3) * 2 + 1];
        };
        auto vf = [&](int, int d, uint32_t (&f)[4]) {
          const int w = (d & 1) * 4;
          f[0] = vw[d >> 1][w];
          f[2] = vw[d >> 1][w + 1];
          f[1] = vw[d >> 1][w + 2];
          f[3] = vw[d >> 1][w + 3];
        };
        tiles(std::integral_constant<int, 1>{}, std::true_type{}, std::true_type{}, kf, vf, ks, vs, pos);
      }
    }

    for (int t = first_of(k.t0, ordinal); t < full_end; t += NG) {
      const int pos = (k.begin + t) * KV8_BLOCK + tt * 16 * MT;
      ok = ok && ring_wait(full + slot, phase, c.err + k.b, stop);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint8_t* src = ring + slot * SLOT;
      uint4 kw[MT][4], vw[MT];  // the values from the slot as they are needed, for want of registers
#pragma unroll
      for (int i = 0; i < 4 * MT; ++i) kw[i / 4][i % 4] = reinterpret_cast<const uint4*>(src + i * 512)[lane];
      float2 sc = *reinterpret_cast<const float2*>(src + 2 * SLICE);
      if (sc.y == 1.0f) {
        // the scale of a block of zeros, too, which says nothing of a magnitude: no weight, no part in the reference
        uint32_t any = 0;
#pragma unroll 1
        for (int i = 0; i < 4 * MT; ++i) {
          const uint4 w = reinterpret_cast<const uint4*>(src + SLICE + i * 512)[lane];
          any |= w.x | w.y | w.z | w.w;
        }
        if (!__any_sync(0xffffffffu, (any & (FMT == HQ_KV8_E4M3 ? 0x7f7f7f7fu : 0xffffffffu)) != 0)) sc.y = 0.f;
      }
      auto release = [&]() {
        __syncwarp();  // every lane has its part: the slot takes the next slice
        ++taken;
        if (issue(slot)) ++issued;
        if (++slot == SLOTS) slot = 0, phase ^= 1;
      };
      auto word = [](const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; };
      auto kf = [&](int j, int s, uint32_t (&f)[4]) {
        // chunk (token half a, d half h) = 2 a + h; word s % 4 of it
        kv8_half4<FMT>(word(kw[j][s >> 2], s & 3), f[0], f[2]);
        kv8_half4<FMT>(word(kw[j][2 + (s >> 2)], s & 3), f[1], f[3]);
      };
      auto vf = [&](int j, int d, uint32_t (&f)[4]) {
        if ((d & 1) == 0) vw[j] = reinterpret_cast<const uint4*>(src + SLICE + (4 * j + (d >> 1)) * 512)[lane];
        kv8_half4<FMT>(word(vw[j], (d & 1) * 2), f[0], f[2]);
        kv8_half4<FMT>(word(vw[j], (d & 1) * 2 + 1), f[1], f[3]);
      };
      const float ks[2] = {sc.x, sc.x}, vs[2] = {sc.y, sc.y};
      constexpr std::integral_constant<int, MT> all{};
      // seen whole by every row?
      if (pos + 16 * MT - 1 <= q_lo && (a.window <= 0 || pos > q_hi - a.window))
        tiles(all, std::false_type{}, std::false_type{}, kf, vf, ks, vs, pos);
      else
        tiles(all, std::true_type{}, std::false_type{}, kf, vf, ks, vs, pos);
      release();
    }

    // after a wait that gave up the warp's part of this task, and of all that follow in the run, is missing
    if (!ok && lane == 0) kv8_err(c, k.b, HQ_DEVERR_TIMEOUT);
    const uint32_t u_next = u + k.units;
    Task k_next = k;
    if (u_next < u1) {
      next_task(u_next, k_next);
      if (warp < NB) load_q(k_next, warp, qv);
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
      const int rr = k.row0 + r;
      if (rr >= rows) return;
      // accumulators are at 2^(P_BIAS - E), the sum at 2^-m: the quotient's exponent
      // a row sees itself at least: no score above -inf means that its query is not finite
      const float f = m == -INFINITY ? NAN : ex2(e - m - P_BIAS), inv = 1.0f / l;
      const int64_t tok = k.s.row0 + rr / a.G;
      const int head = k.h * a.G + rr % a.G;
      E y[4] = {from_float<E>(x.x * inv * f), from_float<E>(x.y * inv * f), from_float<E>(x.z * inv * f), from_float<E>(x.w * inv * f)};
      *reinterpret_cast<uint2*>(static_cast<E*>(a.out) + tok * a.o_tok + head * a.o_head + 4 * lane) =
          *reinterpret_cast<const uint2*>(y);
      if (a.lse != nullptr && lane == 0) a.lse[tok * a.Hq + head] = m == -INFINITY ? NAN : m + log2f(l);
    };
    static_assert(8 % C::WARPS == 0 && C::WARPS % C::OW == 0, "as many of 8 rows to each warp; whole rounds");
    constexpr int RW = 8 / C::WARPS;  // rows 8 nb + warp + i WARPS, elements 4 lane .. 4 lane + 3
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      __syncthreads();  // red is there; the buffer's earlier readers are done
      if (nb == 0 && u_next < u1) stage_q();  // every warp is through with the task's
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float e = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) e = fmaxf(e, red[w * R + 8 * nb + 2 * t4 + i].y);
        f[i] = e == -INFINITY ? 1.f : ex2(e_run[nb][i] - e);
      }
      float m[RW], e[RW], l[RW];
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        m[i] = e[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float4 x = red[w * R + 8 * nb + warp + i * C::WARPS];
          m[i] = fmaxf(m[i], x.x);
          e[i] = fmaxf(e[i], x.y);
        }
        const float mb = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
          const float4 x = red[w * R + 8 * nb + warp + i * C::WARPS];
          l[i] += x.z * ex2(x.x - mb);
        }
      }
      // OW warps at a time add theirs to what the ones before left in their place
#pragma unroll
      for (int w0 = 0; w0 < C::WARPS; w0 += C::OW) {
        if (warp / C::OW == w0 / C::OW) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float* row = obuf + (warp % C::OW * 8 + 2 * t4 + i) * OS + g;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              row[d * 16] = (w0 > 0 ? row[d * 16] : 0.f) + o[nb][d][i] * f[i];
              row[d * 16 + 8] = (w0 > 0 ? row[d * 16 + 8] : 0.f) + o[nb][d][2 + i] * f[i];
            }
          }
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const int r8 = warp + i * C::WARPS, r = 8 * nb + r8;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::OW; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(obuf + (w * 8 + r8) * OS + 4 * lane);
          s.x += x.x;
          s.y += x.y;
          s.z += x.z;
          s.w += x.w;
        }
        if (whole) {
          finish(r, m[i], e[i], l[i], s);
        } else {
          reinterpret_cast<float4*>(part + r * D)[lane] = s;
          if (lane == 0) reinterpret_cast<float4*>(part + R * D)[r] = make_float4(m[i], e[i], l[i], 0.f);
        }
      }
    }
    if (!whole) {
      const uint32_t k0 = u - k.t0;  // the task's first unit
      const int c0 = cta_of(k0), c1 = cta_of(k0 + k.blocks - 1);
      __syncthreads();
      if (threadIdx.x == 0) {
        // the barrier above puts the CTA's writes before this release
        const unsigned int before = atom_add_acq_rel_gpu(a.counters + c0, 1u);
        const bool last = before == static_cast<unsigned int>(c1 - c0);
        if (last) a.counters[c0] = 0u;
        flags[1] = last;
      }
      __syncthreads();
      if (flags[1]) {
        auto piece = [&](int p) { return a.parts + static_cast<size_t>(2 * p + (p == c0)) * PART; };
        auto refs = [&](int r, int p) {
          return p <= c1 ? __ldcg(reinterpret_cast<const float4*>(piece(p) + R * D) + r) : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        };
        for (int r = warp; r < R; r += C::WARPS) {
          // lane i holds the references of pieces c0 + i, c0 + i + 32, ..
          float m = -INFINITY, e = -INFINITY, l = 0.f;
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          // 32 pieces at a time, joined to what was there before; 8 pieces' loads in flight
          for (int p0 = c0; p0 <= c1; p0 += 32) {
            const int n = min(32, c1 - p0 + 1);
            const float4 x = refs(r, p0 + lane);
            float4 y[8];
            auto fetch = [&](int i0) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[i] = i0 + i < n ? __ldcg(reinterpret_cast<const float4*>(piece(p0 + i0 + i) + r * D) + lane)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            };
            fetch(0);
            float m_new = fmaxf(m, x.x), e_new = fmaxf(e, x.y);
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) {
              m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, i));
              e_new = fmaxf(e_new, __shfl_xor_sync(0xffffffffu, e_new, i));
            }
            const float mb = m_new == -INFINITY ? 0.f : m_new, eb = e_new == -INFINITY ? 0.f : e_new;
            const float fo = ex2(e - eb), f = p0 + lane <= c1 ? ex2(x.y - eb) : 0.f;
            l = l * ex2(m - mb) + x.z * ex2(x.x - mb);
            m = m_new;
            e = e_new;
            s.x *= fo;
            s.y *= fo;
            s.z *= fo;
            s.w *= fo;
            for (int i0 = 0; i0 < n; i0 += 8) {
              if (i0 > 0) fetch(i0);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i0 + i);
                s.x += y[i].x * fi;
                s.y += y[i].y * fi;
                s.z += y[i].z * fi;
                s.w += y[i].w * fi;
              }
            }
          }
#pragma unroll
          for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
          finish(r, m, e, l, s);
        }
      }
    }
    if (u_next >= u1) break;
    u = u_next;
    k = k_next;
    ++ordinal;
  }
  // copies that were not waited for (after a wait that gave up) land before the
  // CTA gives its shared memory back
  if (!ok && lane == 0) {
    int never = 0;
    for (; taken < issued; ++taken) ring_wait(full + taken % SLOTS, (taken / SLOTS) & 1, c.err, &never);
  }
}

constexpr int SMEM_MAX = 224 * 1024;  // of an SM: 228 KB less 1 KB for each of up to four CTAs

template <class E, int FMT, int NB, int W>
hq_status launch(Kv8AttnArgs& a, int sms, cudaStream_t st) {
  using C = Cfg<NB, W>;
  static_assert(C::FIXED % 8 == 0 && C::FIXED + HQ_KV8_MAX_BATCH * 8 <= SMEM_MAX / C::CTAS, "shared memory of the largest batch");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "kv8 attention setup");
  static DeviceOnce attrs;
  e = attrs.run(dev, [] {
    return cudaFuncSetAttribute(kv8_attn_kernel<E, FMT, NB, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX / C::CTAS);
  });
  if (e != cudaSuccess) return cuda_fail(e, "kv8 attention setup");
  // units are counted in 32 bits
  if (static_cast<double>(a.c.B) * a.c.Hkv * (a.c.cap / KV8_BLOCK + TASK_UNITS) * 2 >= 4e9) return HQ_ERR_UNSUPPORTED;
  return cuda_status(launch_chained(kv8_attn_kernel<E, FMT, NB, W>, dim3(C::CTAS * sms), C::THREADS, C::FIXED + a.c.B * 8, st, a),
                     "kv8 attention launch");
}

// Rows of a kv head, and rows of a task in eights: up to 24 rows in one task, up to 48 in
// two, which read the pages one after the other, the second mostly from L2.  More go
// to the tcgen05 kernel, whose pages take much the same time for up to 128 rows.  8 kv heads:
// 64 sequences of 1K-8K, 32 rows here 193 us, 48 rows 248, there 49 rows 274, 64 rows 269; one of
// 32K 36, 43, 73, 74; 64 of 100-700 47, 72, 106, 104.  From 64 rows on three tasks would
// take 370 us where batches are large.
constexpr int ROWS_MAX = 48;
int task_eights(int64_t rows) {
  const int n = static_cast<int>((rows + 7) / 8);
  return n <= 3 ? std::max(n, 1) : (n + 1) / 2;
}

// One CTA of 8 warps on an SM, or two of 4.  Where CTAs finish several tasks
// each, one of two streams while the other joins its warps' results (8 kv heads, 128
// sequences of 500-3000: 88 us against 100 us, 64 of 100-700 23 against 28; of
// 1K-16K both 184 us); where tasks are few, twice the pieces are to be joined and
// twice the plans made (one 32K sequence: 8 rows 22.4 us against 20.6 us, 24 rows 40.7
// against 31.7).  A task of more rows takes longer to join (16 windows of 4096, 20 rows:
// 44.4 us against 45.6 us; 8 rows, 16 of 4K-8K: 42.7 against 41.1).
template <class E, int FMT, int NB>
hq_status launch_w(Kv8AttnArgs& a, int sms, cudaStream_t st) {
  if (static_cast<int64_t>(a.c.B) * a.c.Hkv >= (NB == 1 ? 2 * sms : sms / 2))
    return launch<E, FMT, NB, 4>(a, sms, st);
  return launch<E, FMT, NB, 8>(a, sms, st);
}

template <class E, int FMT>
hq_status launch_f(Kv8AttnArgs& a, int sms, cudaStream_t st) {
  switch (task_eights(a.G * a.max_new)) {
    case 1: return launch_w<E, FMT, 1>(a, sms, st);
    case 2: return launch_w<E, FMT, 2>(a, sms, st);
    default: return launch_w<E, FMT, 3>(a, sms, st);
  }
}

constexpr int CTAS = 2;  // most on an SM: HQ_KV8_WS_ZERO holds a counter for each CTA of up to 512 SMs

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

hq_status device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return cuda_status(e, "device query");
}

// Never less for more rows: 25 to 32 rows are two tasks of 16, whose pieces take less than
// those of a task of 24.
size_t attn_workspace(int64_t rows, int sms) {
  const size_t parts = rows > ROWS_MAX ? kv8_attn_tc_parts(rows, sms)
                                       : static_cast<size_t>(2) * CTAS * sms * 8 * (rows > 24 ? 3 : task_eights(rows)) * (D + 4);
  return HQ_KV8_WS_ZERO + parts * sizeof(float);
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
  return hq::attn_workspace(static_cast<int64_t>(Hq / c->Hkv) * max_new, sms);
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
  // the stride of a dimension of one is never used, whatever it says
  if (N == 1) q_tok = o_tok = 0;
  if (Hq == 1) q_head = o_head = 0;
  if (!hq::aligned16(q) || !hq::aligned16(out) || q == out || (q_tok | q_head | o_tok | o_head) % 8) return HQ_ERR_INVALID;
  // scratch is sized from the caller's max_new; fewer rows than that never need more
  int sms = 0;
  const hq_status ds = hq::device_sms(&sms);
  if (ds != HQ_OK) return ds;
  if (!hq::aligned16(ws) || ws_bytes < hq::attn_workspace(static_cast<int64_t>(Hq / c->Hkv) * max_new, sms)) return HQ_ERR_WORKSPACE;
  hq::Kv8AttnArgs a = {};
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
  a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + HQ_KV8_WS_ZERO);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (static_cast<int64_t>(a.G) * max_new > hq::ROWS_MAX) return hq::launch_kv8_attn_tc(a, dtype, sms, s);
  if (dtype == HQ_F16)
    return c->fmt == HQ_KV8_E4M3 ? hq::launch_f<__half, HQ_KV8_E4M3>(a, sms, s) : hq::launch_f<__half, HQ_KV8_INT8>(a, sms, s);
  return c->fmt == HQ_KV8_E4M3 ? hq::launch_f<__nv_bfloat16, HQ_KV8_E4M3>(a, sms, s)
                               : hq::launch_f<__nv_bfloat16, HQ_KV8_INT8>(a, sms, s);
}

}  // extern "C"
