// kv8_attn_tc.cu — attention of many new tokens (prompt chunks, long drafts) over
// the 8-bit block cache on tcgen05 tensor cores: more than 48 rows of a kv head.
//
// The rows of a kv head (its G query heads x the sequence's n new tokens, row
// r = i G + g, so that a page is read once for all of them) are taken NT x 128
// at a time, one TMEM lane a row.  Keys go a page (64 positions) at a time:
//   S = Q K^T    kind::f16, K the page's codes as fp16 (exact), 128 x 64
//   P = 2^(S s_k - m) s_v 2^(m - E + 6) as fp16 (the page's scales in float32)
//   O += P V     kind::f16, P from TMEM (where it takes the place of S), V the
//                page's codes as fp16
// with the two running references m, E of kv8_attn.cu: they are set to the exact
// maxima only when a page's weights of a row sum to more than 2^15, whereupon what
// the row has so far (sum, O) is rescaled.
//
// Warps of a CTA (one CTA an SM, persistent):
//   0-7    softmax: two streams of 128 threads, a row each, with two pages of
//          scores each: one is scored and added while the other's weights are made.
//          NT = 2: the streams are two row tiles over the same pages; NT = 1 (up to
//          128 rows): the same rows, each stream taking every other page, joined at
//          the end
//   8-11   converters, two warps for K and two for V: codes of a page -> fp16 in the 128-byte-swizzled operand
//          layouts, K as [key][d], V as [d][key], both K-major, four stages of each.
//          The page's V order gives a thread 4 keys of one d, which it stores as 8
//          bytes: the keys of 16 stand as t, t+1, t+8, t+9 for t = 0, 2, 4, 6, and
//          P's columns follow the same order
//   12, 13 copies of the pages' codes, K and V (bulk copies, no multicast)
//   14, 15 tcgen05.mma issue, one warp a stream (one for both is the bottleneck: a wait
//          that is met costs it 100 cycles); TMEM allocation
// Bound: two row tiles and 128 keys take 2048 cycles of products, 2048 of
// exponentials and, at 128 bytes a cycle, 3000 of shared memory (256 KB of
// operands, 64 KB converted, 64 KB of codes in and out).
// They take 4200 cycles by the counters: products 49 % of them, the tensor unit with its
// operands' traffic 65 %, exponentials 50 %, shared memory 41 %.  No unit is full, and what
// bounds them (the chain of scores, weights and products with two pages of a stream in
// flight, by the look of it) is not settled.
// Measured: the last 2048 tokens of 16K, 32 query heads over 8: 496 us in a short run,
// 1040 TFLOP/s, 530 us, 972 TFLOP/s, in a long one, where the power limit holds the clock at
// 1.85 GHz; 64
// sequences x 8 tokens x 8 query heads a kv head over 1K-8K: 269 us, one row tile of 64 rows.
// Spills: 16 to 40 bytes a thread.
//
// Work: runs of equal units (pages) as in kv8_attn.cu; pieces of a task that
// CTAs share are joined by the CTA that delivers the last one, in order.
// All waits are bounded (about 1 s): a timeout sets the sequence's error bit and
// the CTA drains its copies and products before it releases TMEM.
#include <cuda_runtime.h>

#include <type_traits>

#include "kv8.cuh"
#include "tc.cuh"

namespace hq {
namespace {

constexpr int TR = 128;                    // rows of a tile
constexpr int STAGES = 4;                  // pages of K, and of V, as operands
constexpr int W_CONV = 8, W_COPY = 12, W_MMA = 14;  // W_COPY: K, W_COPY + 1: V; W_MMA + stream
constexpr int THREADS = 16 * 32;
constexpr float BIAS = 6.0f;               // log2 of the fp16 weight at both references
constexpr float W_TOP = 120.0f;            // of the factor 2^(m - E + BIAS): E stays above m + BIAS - W_TOP (kv8_attn.cu, P_TOP)
constexpr float W_LIMIT = 32768.0f;        // sum of a page's fp16 weights above which the references are set anew
// what a task costs besides its pages, in pages (some 16000 cycles, two thirds of them
// queries, epilogue and the first and last pages' latencies)
// A piece's way through the workspace takes as long as 12 pages: where there is a CTA for
// every task, tasks are cut only if that saves more (8 kv heads, 512 rows: 8 x 128 tokens
// 24 us uncut, 29 cut; 4096 rows of 2048 tokens 53 and 63; 4 x 60 tokens over 2000, where most
// CTAs would stand idle, 60 and 47)
constexpr int UNCUT = 12;
template <int NT>
constexpr int TASK_UNITS = NT == 2 ? 8 : 14;
constexpr uint32_t TMEM_COLS = 512;        // each stream: S 2 x 64 columns (P in the first 32 of each), O 128
constexpr uint32_t TM_S = 0, TM_O = 256;
// fp16, K-major A and B, f32 accumulate
constexpr uint32_t IDESC_QK = idesc_make(0, 0, 0, TR, KV8_BLOCK), IDESC_PV = idesc_make(0, 0, 0, TR, D);
constexpr int HALF = HQ_KV8_V;             // bytes of a page's K (or V) codes

// shared memory (from a 1024-byte aligned base): operands as 128-byte-swizzled
// regions of [128][128 B]
template <int NT>
struct Lay {
  static constexpr int Q = 0;                    // NT x 2 regions (d halves)
  static constexpr int K = Q + NT * 32768;       // stages x 2 regions (d halves): [64 keys][64 d]
  static constexpr int V = K + STAGES * 16384;   // stages: [d][64 keys]
  static constexpr int RAW = V + STAGES * 16384; // codes: slots of a page's K or V
  static constexpr int RK = NT == 2 ? 2 : 4;     // slots of K; as many of V
  static constexpr int RAWS = RAW + 2 * RK * HALF; // the two scales (16 bytes) of each K slot's page
  static constexpr int AUX = RAWS + RK * 16;     // 8 pages x (s_k, s_v, log2 s_v, -); the tail's 64 K and 64 V scales
  static constexpr int BARS = AUX + 8 * 16 + 512;
  static constexpr int MISC = BARS + 48 * 8;     // TMEM base, flags, units of all runs, walk and job
  static constexpr int JOIN = RAW;               // NT = 1: (m, E, l) of stream 1's rows, once the task's copies are done with
  static constexpr int BYTES = MISC + 80 + 144 + 1024;  // with the alignment
};

// Pages [begin, end) that row group grp of a sequence sees, and the positions of its
// first and last row.
struct Span {
  int begin, end, q_lo, q_hi;
};
template <int NT>
__device__ __forceinline__ Span span_of(const Kv8Seq& s, int G, int window, int grp) {
  Span x;
  const int rows = s.n * G, r0 = grp * NT * TR;
  x.q_lo = s.first + r0 / G;
  x.q_hi = s.first + (min(r0 + NT * TR, rows) - 1) / G;
  x.begin = window > 0 ? max(0, x.q_lo + 1 - window) / KV8_BLOCK : 0;
  x.end = x.q_hi / KV8_BLOCK + 1;
  return x;
}
__device__ __forceinline__ int pages_of(const Span& x) { return x.end - x.begin; }

// A task (sequence, kv head, row group) of a CTA's run, [t0, t1) of its pages
// ours, and what the roles need of it.  One thread walks the run; both lie in
// shared memory, for want of registers.
struct Walk {
  int b, h, grp, pages, t0, t1;  // no pages are ours where the run begins behind them
  uint32_t u, u1;                // the task's first unit of ours, the run's end
  uint32_t units;                // ours of the task
  int uncut;                     // a task is one unit
  Kv8Seq s;
  Span sp;
};
struct Job {
  int b, h, row0, rows, tok0;    // rows row0 .. of the kv head's `rows`; the sequence's first row of q
  int first, len;                // position of its first new token, its length
  int page, full_end;            // our first page; complete pages end there, the next one is the tail
  int nt;                        // our pages: 0, the run has no more
  int head, whole;               // the task's first page is ours; all are
  int c0, c1;                    // the CTAs that share the task
};

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int32_t* err, volatile int* stop) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*stop) return false;
    if (global_ns() - t0 > 1000000000ull) {
      atomicOr(reinterpret_cast<unsigned int*>(err), HQ_DEVERR_TIMEOUT);
      *stop = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Whether a page's value codes all stand for zero; a whole warp asks.
template <int FMT>
__device__ __noinline__ bool no_values(const uint8_t* codes) {
  uint32_t any = 0;
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < HALF / 16; i += 32) {
    const uint4 w = reinterpret_cast<const uint4*>(codes)[i];
    any |= w.x | w.y | w.z | w.w;
  }
  return !__any_sync(0xffffffffu, (any & (FMT == HQ_KV8_E4M3 ? 0x7f7f7f7fu : 0xffffffffu)) != 0);
}

// The run's task at k.u (k.t0 of its pages belong to the CTAs before).
template <int NT>
__device__ __noinline__ void enter(const Kv8AttnArgs& a, Walk& k, uint32_t total, Job& j) {
  k.sp = span_of<NT>(k.s, a.G, a.window, k.grp);
  k.pages = pages_of(k.sp);
  k.units = k.uncut ? 1u : min(static_cast<uint32_t>(k.pages + TASK_UNITS<NT> - k.t0), k.u1 - k.u);
  k.t1 = k.uncut ? k.pages : min(k.pages, k.t0 + static_cast<int>(k.units));
  const uint32_t parts = min(total, gridDim.x), run = total / parts, more = total - run * parts;
  // the first `more` runs have a unit more than the others
  auto cta_of = [&](uint32_t u) { return u < more * (run + 1) ? u / (run + 1) : more + (u - more * (run + 1)) / run; };
  j.b = k.b;
  j.h = k.h;
  j.row0 = k.grp * NT * TR;
  j.rows = k.s.n * a.G;
  j.tok0 = k.s.row0;
  j.first = k.s.first;
  j.len = k.s.len;
  j.page = k.sp.begin + k.t0;
  j.full_end = min(k.sp.end, k.s.len / KV8_BLOCK);
  j.nt = max(0, k.t1 - k.t0);
  j.head = k.t0 == 0;
  j.whole = j.nt == k.pages;
  j.c0 = cta_of(k.u - k.t0);
  j.c1 = k.uncut ? j.c0 : cta_of(k.u - k.t0 + k.pages - 1);
}
// The run's next task, or none (j.nt = 0).
template <int NT>
__device__ __noinline__ void next_task(const Kv8AttnArgs& a, Walk& k, uint32_t total, Job& j) {
  j.nt = 0;
  k.u += k.units;
  if (k.u >= k.u1) return;
  k.t0 = 0;
  if (++k.grp * NT * TR >= k.s.n * a.G) {
    k.grp = 0;
    if (++k.h == a.c.Hkv) {
      k.h = 0;
      do {
        ++k.b;
        kv8_seq(a.c, a.cu, a.kv_len, a.N, a.max_new, k.b, false, k.s);
      } while (k.s.n == 0);
    }
  }
  enter<NT>(a, k, total, j);
}

template <class E, int FMT, int NT>
__global__ void __launch_bounds__(THREADS, 1) kv8_attn_tc_kernel(const __grid_constant__ Kv8AttnArgs a) {
  using L = Lay<NT>;
  constexpr int RK = L::RK, ROWS = NT * TR;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BARS);
  // of the slots of codes, of the stages of operands, and [stream * 2 + page % 2]
  uint64_t *rk_full = bars, *rk_empty = bars + 4, *rv_full = bars + 8, *rv_empty = bars + 12, *k_full = bars + 16, *k_empty = bars + 20,
           *v_full = bars + 24, *v_empty = bars + 28, *s_full = bars + 32, *p_full = bars + 36, *o_done = bars + 40;
  uint64_t* drain = bars + 44;
  uint32_t& tmem_sh = *reinterpret_cast<uint32_t*>(sm + L::MISC);
  int* flags = reinterpret_cast<int*>(sm + L::MISC + 4);                  // stop, last
  uint32_t& units_all = *reinterpret_cast<uint32_t*>(sm + L::MISC + 16); // of all runs
  Walk& walk = *reinterpret_cast<Walk*>(sm + L::MISC + 80);
  Job& job = *reinterpret_cast<Job*>(sm + L::MISC + 80 + sizeof(Walk));
  static_assert(sizeof(Walk) + sizeof(Job) <= 144, "their place");
  float* joined = reinterpret_cast<float*>(sm + L::JOIN);                 // [3][TR]
  uint64_t* prefix = reinterpret_cast<uint64_t*>(sm + L::Q);  // the plan, until the queries come
  uint64_t* plan = prefix + HQ_KV8_MAX_BATCH;                 // sums and maxima of each warp
  static_assert((HQ_KV8_MAX_BATCH + 32) * 8 <= 32768, "the plan fits where the queries go");
  const hq_kv8_cache& c = a.c;
  const int B = c.B;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;  // the roles' branches are uniform

  // ---------------------------------------------------------------- plan
  chained();
  // prefix[b]: units (of one kv head) of the sequences before b, in the low half, and
  // their tasks in the high half
  uint64_t carry = 0;
  int longest = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    uint64_t n = 0;
    int top = 0;
    if (b < B) {
      Kv8Seq s;
      kv8_seq(c, a.cu, a.kv_len, a.N, a.max_new, b, blockIdx.x == 0, s);
      const int groups = (s.n * a.G + ROWS - 1) / ROWS;
      for (int i = 0; i < groups; ++i) {
        const int pages = pages_of(span_of<NT>(s, a.G, a.window, i));
        n += 1ull << 32 | static_cast<uint32_t>(pages + TASK_UNITS<NT>);
        top = max(top, pages);
      }
    }
    uint64_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 31) {
      plan[warp] = x;
      plan[16 + warp] = top;
    }
    __syncthreads();
    uint64_t before = carry;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += plan[w];
      carry += plan[w];
      longest = max(longest, static_cast<int>(plan[16 + w]));
    }
    if (b < B) prefix[b] = before + x - n;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    // the units that are dealt out: pages and what a task costs besides them, or whole tasks
    const uint32_t tasks = static_cast<uint32_t>(carry >> 32) * c.Hkv;
    const uint32_t pages = static_cast<uint32_t>(carry) * c.Hkv - tasks * TASK_UNITS<NT>;
    const bool uncut = tasks <= gridDim.x && longest <= UNCUT + static_cast<int>(pages / gridDim.x);
    auto half = [&](uint64_t x) { return uncut ? static_cast<uint32_t>(x >> 32) : static_cast<uint32_t>(x); };
    const uint32_t total = half(carry) * c.Hkv, parts = min(total, gridDim.x);
    job.nt = 0;
    if (blockIdx.x < parts) {
      const uint32_t run = total / parts, more = total - run * parts;
      Walk k;
      k.uncut = uncut;
      k.u = run * blockIdx.x + min(blockIdx.x, more);
      k.u1 = k.u + run + (blockIdx.x < more);
      const uint32_t want = k.u / c.Hkv;
      int lo = 0, hi = B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (half(prefix[mid]) <= want) lo = mid; else hi = mid;
      }
      k.b = lo;
      kv8_seq(c, a.cu, a.kv_len, a.N, a.max_new, lo, false, k.s);
      const uint32_t each = half(lo + 1 < B ? prefix[lo + 1] : carry) - half(prefix[lo]);  // units of a kv head
      uint32_t rel = k.u - half(prefix[lo]) * c.Hkv;
      k.h = rel / each;
      rel -= k.h * each;
      for (k.grp = 0;; ++k.grp) {
        const uint32_t n = uncut ? 1u : pages_of(span_of<NT>(k.s, a.G, a.window, k.grp)) + TASK_UNITS<NT>;
        if (rel < n) break;
        rel -= n;
      }
      k.t0 = rel;
      enter<NT>(a, k, total, job);
      if (job.nt == 0) next_task<NT>(a, k, total, job);  // the run begins behind a task's pages
      walk = k;
      units_all = total;
    }
  }
  __syncthreads();
  if (job.nt == 0) return;

  // ---------------------------------------------------------------- setup
  if (threadIdx.x == 0) {
    for (int i = 0; i < RK; ++i) {
      mbar_init(rk_full + i, 1);
      mbar_init(rk_empty + i, 64);
      mbar_init(rv_full + i, 1);
      mbar_init(rv_empty + i, 64);
    }
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(k_full + i, 64);
      mbar_init(k_empty + i, NT);
      mbar_init(v_full + i, 64);
      mbar_init(v_empty + i, NT);
    }
    for (int i = 0; i < 2; ++i) mbar_init(drain + i, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(o_done + i, 1);
    }
    flags[0] = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) {
    tmem_alloc(&tmem_sh, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  const uint32_t base = smem_u32(sm);
  volatile int* stop = flags;
  float* aux = reinterpret_cast<float*>(sm + L::AUX);
  float* tail_sc = aux + 8 * 4;  // [K, V][64]

  // running uses of each barrier, kept by the roles that wait on it
  int n_raw = 0;                  // copied pages (copy warps), those before the task's (converters)
  int n_page = 0;                 // pages before the task's (converters, MMA, the softmax's scales)
  int n_mine = 0;                 // pages of the stream (softmax, MMA)
  bool ok = true;
  auto takes = [&](int g, int t) { return NT == 2 || (t & 1) == g; };

  while (true) {
    const size_t bh = static_cast<size_t>(job.b) * c.Hkv + job.h;
    const int rows = job.rows, nt = job.nt, page0 = job.page;
    const int full = min(nt, job.full_end - page0);  // our complete pages; the tail may follow
    int32_t* err = c.err + job.b;

    // ---------------------------------------------------------- queries -> shared memory
    // half a warp a row, 16 bytes a lane; every load of the warp's 32 rows in flight at once
    float qmul = a.scale;
    if (warp < 8) {
      const int r0 = (warp & 3) * 32, tile = NT == 2 ? warp >> 2 : 0, ch = lane & 15;  // stream 1 of NT = 1: the same rows
      uint4 v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int rr = job.row0 + tile * TR + r0 + 2 * i + (lane >> 4);
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (rr < rows)
          v[i] = reinterpret_cast<const uint4*>(static_cast<const E*>(a.q) + static_cast<int64_t>(job.tok0 + rr / a.G) * a.q_tok +
                                                static_cast<int64_t>(job.h * a.G + rr % a.G) * a.q_head)[ch];
      }
      float* unit = reinterpret_cast<float*>(sm + L::RAW) + warp * 32;  // the copies' place: they wait for the queries
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4);
        if (IsBf16<E>::value) {
          // bf16 rows become fp16 at a power of two that brings their largest value to [2^14, 2^15)
          E e[8];
          *reinterpret_cast<uint4*>(e) = v[i];
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(to_float(e[j])) & 0x7fffffffu);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          float inv = 1.0f, u = 1.0f;
          if (m != 0 && m < 0x7f800000u) {
            const int ex = max(static_cast<int>(m >> 23) - 127 - 14, -126);
            u = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
            inv = ex == -126 ? 0x1p126f : __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
          }
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = pack_f16x2(to_float(e[2 * j]) * inv, to_float(e[2 * j + 1]) * inv);
          v[i] = make_uint4(w[0], w[1], w[2], w[3]);
          if (ch == 0) unit[r] = u;
        }
        if (NT == 2 || warp < 4)
          sts128(base + L::Q + tile * 32768 + (ch >> 3) * 16384 + (r0 + r) * 128 + (((ch & 7) ^ (r & 7)) << 4), v[i].x, v[i].y, v[i].z, v[i].w);
      }
      if (IsBf16<E>::value) {
        __syncwarp();
        qmul *= unit[lane];
      }
      fence_proxy_async_smem();
    }
    __syncthreads();

    if (warp == W_COPY || warp == W_COPY + 1) {
      // -------------------------------------------------------- copies
      // 32 pages looked up at a time, and the next 32 while these are copied
      const int which = warp - W_COPY;
      uint64_t* slot_empty = which ? rv_empty : rk_empty;
      uint64_t* slot_full = which ? rv_full : rk_full;
      const int p_begin = page0, p_end = page0 + full;
      auto look_up = [&](int p) { return p + lane < p_end ? reinterpret_cast<uint64_t>(kv8_page(c, bh, p + lane)) : 0ull; };
      uint64_t next = look_up(p_begin);
      for (int p = p_begin; ok && p < p_end; p += 32) {
        const uint64_t now = next;
        next = look_up(p + 32);
        const int m = min(32, p_end - p);
        for (int i = 0; ok && i < m; ++i, ++n_raw) {
          const int sl = n_raw % RK;
          const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, now, i));
          if (n_raw >= RK) ok = wait_for(slot_empty + sl, (n_raw / RK - 1) & 1, err, stop);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(slot_full + sl, which ? HALF : HALF + 16);
            bulk_g2s(sm + L::RAW + (which * RK + sl) * HALF, page + which * HQ_KV8_V, HALF, slot_full + sl);
            if (!which) bulk_g2s(sm + L::RAWS + sl * 16, page + HQ_KV8_KSCALE, 16, slot_full + sl);
          }
        }
      }
    } else if (warp >= W_CONV && warp < W_COPY) {
      // -------------------------------------------------------- converters
      const int cw = (warp - W_CONV) & 1, ct = cw * 32 + lane;  // warp of two, thread of 64
      const int g = lane >> 2, t4 = lane & 3;
      auto await = [&](uint64_t* bar, int parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1))) return true;  // each lane has acquired the phase itself
        ok = wait_for(bar, parity & 1, err, stop);
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      auto convert = [&](auto which) {
        constexpr bool VAL = decltype(which)::value;  // values, else keys
        uint64_t* slot_full = VAL ? rv_full : rk_full;
        uint64_t* slot_empty = VAL ? rv_empty : rk_empty;
        uint64_t* st_full = VAL ? v_full : k_full;
        uint64_t* st_empty = VAL ? v_empty : k_empty;
        // where the thread's part of a stage goes.  K: 16 d of one key, two 16-byte
        // operand chunks; V: 4 keys of each of 4 d, 8 bytes each
        auto put = [&](uint32_t dst, int e, const uint32_t (&y)[8]) {
          if (VAL) {  // 512 bytes of codes: 16 keys (e / 4) x 32 d (e % 4)
            const uint32_t row = dst + ((e & 3) * 32 + g) * 128 + ((((e >> 2) * 2 + (t4 >> 1)) ^ g) << 4) + (t4 & 1) * 8;
            sts64(row, y[0], y[1]);
            sts64(row + 8 * 128, y[2], y[3]);
            sts64(row + 16 * 128, y[4], y[5]);
            sts64(row + 24 * 128, y[6], y[7]);
          } else {    // 8 keys (e / 2) x 64 d (e % 2)
            const uint32_t row = dst + (e & 1) * 8192 + ((e >> 1) * 8 + g) * 128;
            sts128(row + (((2 * t4) ^ g) << 4), y[0], y[1], y[2], y[3]);
            sts128(row + (((2 * t4 + 1) ^ g) << 4), y[4], y[5], y[6], y[7]);
          }
        };
        for (int t = 0; t < full; ++t) {
          const int T = n_page + t, st = T % STAGES, sl = (n_raw + t) % RK;
          if (!await(slot_full + sl, (n_raw + t) / RK)) return;
          const uint4* src = reinterpret_cast<const uint4*>(sm + L::RAW + ((VAL ? RK : 0) + sl) * HALF) + cw * 8 * 32 + lane;
          uint4 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = src[i * 32];
          float2 sc = VAL ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2*>(sm + L::RAWS + sl * 16);
          // also the scale of a block of zeros, which says nothing of a magnitude: no weight, no part in the reference
          if (!VAL && cw == 0 && sc.y == 1.0f && no_values<FMT>(kv8_page(c, bh, page0 + t) + HQ_KV8_V)) sc.y = 0.f;
          mbar_arrive(slot_empty + sl);
          // The stage is free once the page four before has been scored (K) or added (V).
          // Scoring that page took the place of the one four before it in its stream at
          // least, so that the scales of eight pages before have been used.
          if (T >= STAGES && !await(st_empty + st, T / STAGES - 1)) return;
          if (!VAL && ct == 0)
            *reinterpret_cast<float4*>(aux + (T & 7) * 4) = make_float4(sc.x, sc.y, lg2_approx(sc.y), 0.f);
          const uint32_t dst = base + (VAL ? L::V : L::K) + st * 16384;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t y[8];
            kv8_half4<FMT>(x[i].x, y[0], y[1]);
            kv8_half4<FMT>(x[i].y, y[2], y[3]);
            kv8_half4<FMT>(x[i].z, y[4], y[5]);
            kv8_half4<FMT>(x[i].w, y[6], y[7]);
            put(dst, cw * 8 + i, y);
          }
          fence_proxy_async_smem();
          mbar_arrive(st_full + st);
        }
        if (full < nt) {
          // the incomplete block, in 16 bits from where it lies
          const int T = n_page + full, st = T % STAGES, half = (page0 + full) & 1;
          if (T >= STAGES && !await(st_empty + st, T / STAGES - 1)) return;
          const uint32_t dst = base + (VAL ? L::V : L::K) + st * 16384;
          const uint4* src = reinterpret_cast<const uint4*>((VAL ? c.tail_v : c.tail_k) + (bh * 2 + half) * KV8_BLOCK * D);
          const float* ts = c.tail_scale + (bh * 2 + VAL) * HQ_KV8_TAIL + half * KV8_BLOCK;
          const int held = job.len - (page0 + full) * KV8_BLOCK;  // rows of the block
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            uint32_t y[4][8];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int e = cw * 8 + i * 4 + w;
              *reinterpret_cast<uint4*>(y[w]) = src[(e * 32 + lane) * 2];
              *reinterpret_cast<uint4*>(y[w] + 4) = src[(e * 32 + lane) * 2 + 1];
            }
            if (VAL) {
              // the 16 rows at their own magnitude; past the length nothing is seen, and no value counts for a reference
              const int r0 = (cw * 2 + i) * 16 + 2 * t4;
#pragma unroll
              for (int z = 0; z < 2; ++z) {  // rows r0, r0 + 1; those 8 behind
                uint32_t top = 0;
#pragma unroll
                for (int w = 0; w < 16; ++w) top = kv8_top2(top, y[w / 4][w % 4 * 2 + z]);
#pragma unroll
                for (int o = 4; o < 32; o *= 2) top = kv8_top2(top, __shfl_xor_sync(0xffffffffu, top, o));
                const TailUp up(top);
#pragma unroll
                for (int w = 0; w < 16; ++w) y[w / 4][w % 4 * 2 + z] = up(y[w / 4][w % 4 * 2 + z]);
                if (g < 2) {
                  const int r = r0 + 8 * z + g;
                  tail_sc[64 + r] = r < held ? kv8_tail_vscale(ts[r], top >> g * 16 & 0x7fffu) : 0.0f;
                }
              }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) put(dst, cw * 8 + i * 4 + w, y[w]);
          }
          if (!VAL) {
            if (ct == 0) *reinterpret_cast<float4*>(aux + (T & 7) * 4) = make_float4(1.f, 1.f, 0.f, 0.f);
            tail_sc[ct] = ct < held ? ts[ct] : 1.0f;
            // the block is scored once the scales of its values are there, too (a wait for them
            // by the softmax warps cost every page's code: prompt chunk 542 us against 502)
            if (!await(v_full + st, T / STAGES)) return;
          }
          fence_proxy_async_smem();
          mbar_arrive(st_full + st);
        }
      };
      if (ok) {
        if (warp < W_CONV + 2) convert(std::false_type{});
        else convert(std::true_type{});
      }
      n_raw += full;
      n_page += nt;
    } else if (warp >= W_MMA) {
      // -------------------------------------------------------- MMA issue
      // the whole warp, in uniform control flow; its leader issues
      const int g = warp - W_MMA;
      const uint32_t leader = elect_leader();
      auto await = [&](uint64_t* bar, int parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1))) return true;  // each lane has acquired the phase itself
        ok = wait_for(bar, parity & 1, err, stop);
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      // A stream's page j takes the place of page j - 2, once that has been added.  A
      // page's operand is free when every stream that takes it is done with it.
      auto score = [&](int t, int j, bool again) {
        const int T = n_page + t, st = T % STAGES, sb = 2 * g + (j & 1);
        if ((again && !await(o_done + sb, (j >> 1) - 1)) || !await(k_full + st, T / STAGES)) return;
        tc_fence_after();
        const uint32_t Qs = base + L::Q + (NT == 2 ? g * 32768 : 0), Ks = base + L::K + st * 16384;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_f16_warp(leader, tmem + TM_S + 64 * sb, sdesc_sw128(Qs + (kk >> 2) * 16384 + 32 * (kk & 3), 16, 1024),
                        sdesc_sw128(Ks + (kk >> 2) * 8192 + 32 * (kk & 3), 16, 1024), IDESC_QK, kk > 0);
        umma_commit_warp(leader, s_full + sb);
        umma_commit_warp(leader, k_empty + st);
      };
      constexpr int STEP = NT == 2 ? 1 : 2;
      const int t0 = NT == 2 ? 0 : g;
      if (ok && t0 < nt) score(t0, n_mine, false);
      if (ok && t0 + STEP < nt) score(t0 + STEP, n_mine + 1, false);
      for (int t = t0; ok && t < nt; t += STEP, ++n_mine) {
        const int T = n_page + t, st = T % STAGES, j = n_mine, sb = 2 * g + (j & 1);
        if (!await(p_full + sb, j >> 1) || !await(v_full + st, T / STAGES)) break;
        tc_fence_after();
        const uint32_t Vs = base + L::V + st * 16384;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ta_warp(leader, tmem + TM_O + 128 * g, tmem + TM_S + 64 * sb + 8 * kk, sdesc_sw128(Vs + 32 * kk, 16, 1024),
                           IDESC_PV, t > t0 || kk > 0 ? 1u : 0u);
        umma_commit_warp(leader, o_done + sb);
        umma_commit_warp(leader, v_empty + st);
        if (t + 2 * STEP < nt) score(t + 2 * STEP, j + 2, true);
      }
      n_page += nt;
    } else {
      // -------------------------------------------------------- softmax
      const int g = warp >> 2, r = threadIdx.x & 127;
      const int rr = job.row0 + (NT == 2 ? g * TR : 0) + r;  // row of the (sequence, kv head)
      const bool real = rr < rows;
      const int qpos = job.first + rr / a.G;
      const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t orow = trow + TM_O + 128 * g;
      // rows past the last have zero queries and see every key; their references
      // start at 1.  A warp without a row only keeps the barriers going.
      float m = real ? -INFINITY : 0.f, e = real ? -INFINITY : 0.f, l = 0.f;
      const bool idle = !__any_sync(0xffffffffu, real);
      int taken = 0;  // pages of the task
      for (int t = 0; t < nt; ++t) {
        if (!takes(g, t)) continue;
        const int j = n_mine, sb = 2 * g + (j & 1);
        const uint32_t srow = trow + TM_S + 64 * sb;
        ok = ok && wait_for(s_full + sb, (j >> 1) & 1, err, stop);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        ++n_mine;
        ++taken;
        if (idle) {
          mbar_arrive(p_full + sb);
          continue;
        }
        float x[64];
        auto load = [&]() {
          tmem_ld32f(srow, x);
          tmem_ld32f(srow + 32, x + 32);
          tmem_wait_ld();
        };
        load();
        const bool tail = t >= full;
        const float4 sc = *reinterpret_cast<const float4*>(aux + ((n_page + t) & 7) * 4);  // s_k, s_v, log2 s_v, -
        // columns [lo, hi] of the page are seen by this row
        const int hi = real ? qpos - (page0 + t) * KV8_BLOCK : KV8_BLOCK, lo = real && a.window > 0 ? hi - a.window + 1 : 0;
        const bool seen = __all_sync(0xffffffffu, !tail && hi >= KV8_BLOCK - 1 && lo <= 0);  // all columns, by 16-bit rows none
        const float mul = qmul * sc.x;
        // the scores (exponents of 2) of a page that is not seen whole, masked ones -inf
        auto mask = [&]() {
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const float f = tail ? qmul * tail_sc[i] : mul;
            x[i] = i >= lo && i <= hi ? x[i] * f : -INFINITY;
          }
        };
        // The references anew, from the exact maximum of the page; sum and O are rescaled.
        auto renew = [&]() {
          load();
          float mt = -INFINITY, et = -INFINITY;  // largest score, largest score + log2(value scale); NaN is passed over
          if (seen) {
#pragma unroll
            for (int i = 0; i < 64; ++i) mt = fmaxf(mt, x[i] * mul);
          } else {
            mask();
#pragma unroll
            for (int i = 0; i < 64; ++i) mt = fmaxf(mt, x[i]);
          }
          if (tail) {
            // each position has its own scale: those that the row does not see are at -inf
#pragma unroll
            for (int i = 0; i < 64; ++i) et = fmaxf(et, x[i] + lg2_approx(tail_sc[64 + i]));
          } else {
            et = mt + sc.z;
          }
          // a page's factor times its scale is finite, too
          const float low = (tail ? 0.f : fmaxf(sc.z, 0.f)) + (BIAS - W_TOP);
          const float m_new = fmaxf(m, mt), e_new = fmaxf(fmaxf(e, et), m_new + low);
          const float mb = m_new == -INFINITY ? 0.f : m_new, eb = e_new == -INFINITY ? 0.f : e_new;
          const float ao = ex2(e - eb);
          l *= ex2(m - mb);
          m = m_new;
          e = e_new;
          if (taken > 1) {
            // the page before may still be being added
            ok = wait_for(o_done + (sb ^ 1), ((j - 1) >> 1) & 1, err, stop);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
#pragma unroll 1
            for (int c4 = 0; c4 < 4; ++c4) {
              uint32_t y[32];
              tmem_ld32(orow + 32 * c4, y);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * ao);
              tmem_st32(orow + 32 * c4, y);
            }
            tmem_wait_st();
          }
          load();
        };
        bool fresh = __any_sync(0xffffffffu, m == -INFINITY);
        if (fresh) renew();
        uint32_t pk[32];
        float s0, s1;  // sums of the fp16 weights and of the softmax's
        while (true) {
          const float mref = m == -INFINITY ? 0.f : m;
          // Weights of a page that is seen whole take the value scale into the
          // exponent, and their sum is divided by it: a product less per weight.
          // (The logarithm's error, 2^-22, goes to the page's weights and not to their sum.)
          // Not where it is so small that weights would underflow.
          const float off = BIAS - e + sc.z, lw = m + off;
          if (__all_sync(0xffffffffu, seen && lw > -60.f)) {
            const uint64_t mul2 = f32x2(mul, mul), off2 = f32x2(off, off);
            uint64_t a0 = 0, a1 = 0;
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              const float2 z = f32x2_split(f32x2_fma(f32x2(x[i], x[i + 1]), mul2, off2));
              const float y0 = ex2(z.x), y1 = ex2(z.y);
              uint64_t& acc = i & 2 ? a1 : a0;
              acc = f32x2_add(acc, f32x2(y0, y1));
              pk[i / 2] = pack_f16x2(y0, y1);
            }
            const float2 b0 = f32x2_split(f32x2_add(a0, a1));
            s0 = b0.x + b0.y;
            s1 = s0 * ex2(-lw);
          } else {
            const float ef = e == -INFINITY ? 0.f : ex2(m - e + BIAS), w = ef * sc.y;
            if (seen) {
#pragma unroll
              for (int i = 0; i < 64; ++i) x[i] *= mul;
            } else {
              mask();
            }
            s0 = s1 = 0.f;
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              float y0 = ex2(x[i] - mref), y1 = ex2(x[i + 1] - mref);
              s1 += y0 + y1;
              // a scale that is NaN stays behind the mask
              y0 = x[i] == -INFINITY ? 0.f : tail ? y0 * ef * tail_sc[64 + i] : y0 * w;
              y1 = x[i + 1] == -INFINITY ? 0.f : tail ? y1 * ef * tail_sc[64 + i + 1] : y1 * w;
              s0 += y0 + y1;
              pk[i / 2] = pack_f16x2(y0, y1);
            }
          }
          if (!__any_sync(0xffffffffu, !(s0 <= W_LIMIT)) || fresh) break;  // also an infinity or NaN
          renew();
          fresh = true;
        }
        // P's columns: pairs of keys, those of 16 in V's order 0 1 8 9, 2 3 10 11, 4 5 12 13, 6 7 14 15
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = pk[(i & 24) + (i & 1) * 4 + ((i & 7) >> 1)];
        tmem_st32(srow, w);
        tmem_wait_st();
        l += s1;
        tc_fence_before();
        mbar_arrive(p_full + sb);
      }
      n_page += nt;
      if (taken > 0 && ok) ok = wait_for(o_done + 2 * g + ((n_mine - 1) & 1), ((n_mine - 1) >> 1) & 1, err, stop);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();

      // ------------------------------------------------------ the CTA's piece of the task
      const bool whole = job.whole;
      auto o_cols = [&](int c4, float (&x)[32]) {
        tmem_ld32f(orow + 32 * c4, x);
        tmem_wait_ld();
      };
      float* swap = reinterpret_cast<float*>(sm + L::K);  // [column][row]: the keys are done with
      if (NT == 1) {
        // stream 1 hands its rows to stream 0, once both streams are through with the
        // keys and every code of the task has been converted
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (g == 1) {
          joined[r] = m;
          joined[TR + r] = taken > 0 ? e : -INFINITY;
          joined[2 * TR + r] = l;
        }
        if (g == 1 && ok && taken > 0 && !idle) {
#pragma unroll 1
          for (int c4 = 0; c4 < 4; ++c4) {
            float x[32];
            o_cols(c4, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) swap[(32 * c4 + i) * TR + r] = x[i];
          }
        }
        asm volatile("bar.sync 2, 256;" ::: "memory");
      }
      // pieces: slot 2 cta (+ 1 for the task's first), [stream's rows][column][row] and (m, E, l)
      constexpr int PIECE = TR * (D + 3);
      const int q = NT == 2 ? g : 0;
      float* part = a.parts + (static_cast<size_t>(2 * blockIdx.x + job.head) * NT + q) * PIECE;
      const int c0 = job.c0, c1 = job.c1;
      const bool owner = NT == 2 || g == 0;  // threads that hold the piece's rows
      float m2 = -INFINITY, e2 = -INFINITY, l2 = 0.f;
      if (NT == 1 && owner && nt > 1) {
        m2 = joined[r];
        e2 = joined[TR + r];
        l2 = joined[2 * TR + r];
      }
      const float mj = fmaxf(m, m2), ej = fmaxf(e, e2);
      const float mb = mj == -INFINITY ? 0.f : mj, eb = ej == -INFINITY ? 0.f : ej;
      const float lj = l * ex2(m - mb) + l2 * ex2(m2 - mb);
      const float f1 = ej == -INFINITY ? 1.f : ex2(e - eb), f2 = ej == -INFINITY ? 1.f : ex2(e2 - eb);
      auto write = [&](float m, float e, float l, auto cols) {  // the row's output from its accumulators
        // accumulators are at 2^(BIAS - E), the sum at 2^-m
        // a row sees itself at least: no score above -inf means that its query is not finite
        const float f = m == -INFINITY ? NAN : ex2(e - m - BIAS), inv = 1.0f / l;
        const int64_t tok = job.tok0 + rr / a.G;
        const int head = job.h * a.G + rr % a.G;
        E* dst = static_cast<E*>(a.out) + tok * a.o_tok + head * a.o_head;
#pragma unroll 1
        for (int c4 = 0; c4 < 4; ++c4) {
          float x[32];
          cols(c4, x);
          if (real) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              E y[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) y[z] = from_float<E>(x[i + z] * inv * f);
              *reinterpret_cast<uint4*>(dst + 32 * c4 + i) = *reinterpret_cast<const uint4*>(y);
            }
          }
        }
        if (real && a.lse != nullptr) a.lse[tok * a.Hq + head] = m == -INFINITY ? NAN : m + log2f(l);
      };
      if (owner && ok && !idle) {
        auto cols = [&](int c4, float (&x)[32]) {
          o_cols(c4, x);
          if (NT == 1) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = x[i] * f1 + (nt > 1 ? swap[(32 * c4 + i) * TR + r] * f2 : 0.f);
          }
        };
        if (whole) {
          write(mj, ej, lj, cols);
        } else {
#pragma unroll 1
          for (int c4 = 0; c4 < 4; ++c4) {
            float x[32];
            cols(c4, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) __stcg(part + (32 * c4 + i) * TR + r, x[i]);
          }
          __stcg(part + D * TR + r, mj);
          __stcg(part + (D + 1) * TR + r, ej);
          __stcg(part + (D + 2) * TR + r, lj);
        }
      }
      if (!whole) {
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (threadIdx.x == 0) {
          // the barrier puts the CTA's writes before this release
          const unsigned int before = atom_add_acq_rel_gpu(a.counters + c0, 1u);
          const bool last = before == static_cast<unsigned int>(c1 - c0);
          if (last) a.counters[c0] = 0u;
          flags[1] = last;
        }
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (flags[1] && owner && ok && !idle) {
          auto piece = [&](int p) { return a.parts + (static_cast<size_t>(2 * p + (p == c0)) * NT + q) * PIECE; };
          float mm = -INFINITY, ee = -INFINITY, ll = 0.f;
          for (int p = c0; p <= c1; ++p) {
            mm = fmaxf(mm, __ldcg(piece(p) + D * TR + r));
            ee = fmaxf(ee, __ldcg(piece(p) + (D + 1) * TR + r));
          }
          const float mmb = mm == -INFINITY ? 0.f : mm, eeb = ee == -INFINITY ? 0.f : ee;
          for (int p = c0; p <= c1; ++p) ll += __ldcg(piece(p) + (D + 2) * TR + r) * ex2(__ldcg(piece(p) + D * TR + r) - mmb);
          write(mm, ee, ll, [&](int c4, float (&x)[32]) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0.f;
            for (int p = c0; p <= c1; ++p) {
              const float* src = piece(p) + 32 * c4 * TR + r;
              const float f = ex2(__ldcg(piece(p) + (D + 1) * TR + r) - eeb);
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] += __ldcg(src + i * TR) * f;
            }
          });
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    __syncthreads();  // the task's shared and tensor memory is free
    tc_fence_after();
    if (threadIdx.x == 0) {
      next_task<NT>(a, walk, units_all, job);
      // after a wait that gave up: the sequences of the tasks that are not begun are marked, and
      // their pieces counted, so that the counters go back to zero all the same
      if (*stop) {
        for (; job.nt != 0; next_task<NT>(a, walk, units_all, job)) {
          kv8_err(c, job.b, HQ_DEVERR_TIMEOUT);
          if (!job.whole && atom_add_acq_rel_gpu(a.counters + job.c0, 1u) == static_cast<unsigned int>(job.c1 - job.c0))
            a.counters[job.c0] = 0u;
        }
      }
    }
    __syncthreads();
    if (job.nt == 0) break;
  }

  // Products and copies that were not waited for (only after a wait that gave up)
  // end before TMEM and shared memory are given back.
  if (warp >= W_MMA) {
    umma_commit_warp(elect_leader(), drain + (warp - W_MMA));
    int never = 0;
    wait_for(drain + (warp - W_MMA), 0, c.err, &never);
  }
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
  if ((warp == W_COPY || warp == W_COPY + 1) && lane == 0 && *stop) {
    int never = 0;
    for (int i = max(0, n_raw - RK); i < n_raw; ++i) wait_for((warp == W_COPY ? rk_full : rv_full) + i % RK, (i / RK) & 1, c.err, &never);
  }
}

template <class E, int FMT, int NT>
hq_status launch(const Kv8AttnArgs& a, int sms, cudaStream_t st) {
  using L = Lay<NT>;
  static_assert(L::BYTES <= 227 * 1024, "shared memory of a CTA");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "kv8 attention setup");
  static DeviceOnce attrs;
  e = attrs.run(dev, [] {
    return cudaFuncSetAttribute(kv8_attn_tc_kernel<E, FMT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  });
  if (e != cudaSuccess) return cuda_fail(e, "kv8 attention setup");
  // units are counted in 32 bits
  const double groups = static_cast<double>(a.G) * a.max_new / (NT * TR) + 1;
  if (groups * a.c.B * a.c.Hkv * (a.c.cap / KV8_BLOCK + TASK_UNITS<NT>) >= 4e9) return HQ_ERR_UNSUPPORTED;
  return cuda_status(launch_chained(kv8_attn_tc_kernel<E, FMT, NT>, dim3(sms), THREADS, L::BYTES, st, a), "kv8 attention launch");
}

template <class E, int FMT>
hq_status launch_f(const Kv8AttnArgs& a, int sms, cudaStream_t st) {
  // one row tile with two streams over the keys, or two row tiles
  return a.G * static_cast<int64_t>(a.max_new) <= TR ? launch<E, FMT, 1>(a, sms, st) : launch<E, FMT, 2>(a, sms, st);
}

}  // namespace

// floats of the workspace's pieces for `rows` rows of a kv head
size_t kv8_attn_tc_parts(int64_t rows, int sms) { return static_cast<size_t>(2) * sms * (rows <= TR ? 1 : 2) * TR * (D + 3); }

hq_status launch_kv8_attn_tc(const Kv8AttnArgs& a, int dtype, int sms, cudaStream_t st) {
  if (dtype == HQ_F16)
    return a.c.fmt == HQ_KV8_E4M3 ? launch_f<__half, HQ_KV8_E4M3>(a, sms, st) : launch_f<__half, HQ_KV8_INT8>(a, sms, st);
  return a.c.fmt == HQ_KV8_E4M3 ? launch_f<__nv_bfloat16, HQ_KV8_E4M3>(a, sms, st)
                                : launch_f<__nv_bfloat16, HQ_KV8_INT8>(a, sms, st);
}

}  // namespace hq
