// Attention of ragged rows over a paged cache held in 8 bits.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - m),  lse = m + log sum_t p_t
// over the tokens t that a row sees: t < hi, hi = kv_len (causal: kv_len - n + j + 1 for row j of n),
// and t >= hi - window with a window.  A row that sees nothing gets 0 and lse = -inf.
//
// The cache's e4m3 elements go into the tensor cores as they are; what would have to be converted are the queries
// and the probabilities, of which there are few.  A step takes 128 tokens of one key/value head and N row-heads
// (the query heads of that head times the request's rows) and works transposed, tokens (then dimensions) on the
// 128-wide side:
//   S^T [token, row-head] = K Q^T,   O^T [dimension, row-head] += V^T P^T
// with Q and P as sums of e5m2 terms, each the top byte of the fp16 value that is left: 3 terms hold the 8 bits of
// a bf16 query, 4 the 11 bits of an fp16 one.  The terms of Q follow one another into the same sum, those of P lie side
// by side in N (its operand of values is read once) and are added at the end.  A block's scales touch no element:
// the keys' multiplies the scores of its tokens, the values' their probabilities before they are split.
//
// The range of e5m2 (2^15.8 down to 2^-16) is what P is kept in: the running reference of a row-head is the maximum of
// score + log2(value scale), put at 2^11.5, and moves when a product passes 2^15.5.  What lies below 2^-28 of the
// reference is rounded away; a million such tokens would make 2^-8.
//
// Rounding: scores, sums and outputs are fp32; probabilities are rounded to fp16 and then, for bf16 queries, to 9 bits
// (2^-10 of each, as bf16 outputs are), for fp16 queries not at all.
//
// The steps of all units (request, key/value head, tile of N row-heads) lie in one row, cut into as many equal pieces as
// CTAs fit on the GPU: lengths need not be alike for all to end together, and one long request fills the GPU by
// itself.  A unit that is cut leaves its pieces' sums in a workspace, where join_kernel adds them in order.
//
// Measured (one GB300): one request of 131071 tokens with 8 rows, 32 query and 8 key/value heads of 128 dimensions, 85 us
// (40 us of reading at the memory's rate); 64 requests of 512 to 4096 tokens with 1 to 8 rows 141 us (46); 256 requests
// of up to 16384 tokens, heads of 64 dimensions, 672 us (359).  Bound by a step's chain (scores out of tensor memory,
// exponents, terms, stores, products) with two CTAs an SM, and by what a piece costs before and after its steps.  One
// group of four warps on all row-heads took 112, 198 and 822 us.
//
// Warps 0-3 and 4-7: half of the row-heads each; a thread has a token of S^T (scales, mask, exponentials, terms of P),
// then a dimension of O^T.  Warp 8 brings keys and values by bulk copies into a ring, looking up pages a step ahead.
// Warp 9 issues the products: S of the next step before P V of this one.
#include <type_traits>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kTokens = 128;
constexpr int kThreads = 10 * 32;
constexpr float kTop = 11.5f, kBar = 15.5f;      // log2 of where the largest product is put, and may rise to
constexpr float kNone = 1e30f;                   // the offset of a row-head without a reference: every score passes

template <int DT, int D, int N>
struct Shape {
  static constexpr int kTerms = DT == DSPARK_BF16 ? 3 : 4;
  static constexpr int kCtas = N <= 32 ? 2 : 1;                         // on an SM together
  static constexpr int kSlot = kTokens * D;
  static constexpr int kP = kTerms * N * kTokens, kQ = kTerms * N * D;
  static constexpr int kRoom = (kCtas == 2 ? 109 : 216) * 1024 - kP - kQ;
  static constexpr int kSlots = kRoom / kSlot < 16 ? kRoom / kSlot : 16;
  static constexpr int kOffP = kSlots * kSlot, kOffQ = kOffP + kP, kOffSh = kOffQ + kQ;
  static constexpr int kColumns = (2 + kTerms) * N;                     // of tensor memory: S twice, O's terms
  static constexpr int kAlloc = kColumns <= 128 ? 128 : (kColumns <= 256 ? 256 : 512);
  static constexpr int kPartial = N * (D + 2);                          // floats of a piece's sums
  static_assert(kSlots >= 4, "the look at values of an edge relies on it");
};

template <int SLOTS, int N>
struct Shared {
  uint64_t full[SLOTS], empty[SLOTS], s_full[2], p_full, o_done, q_ready, drain;
  alignas(16) float R[N], z[N];
  float ref[N], factor[N], most[4][N], sum[4][N];
  int hi[N];
  int64_t scan[kThreads / 32];
  int64_t begin_request, begin_at, total;
  uint32_t tmem;
  int abort, skip, odd;
};

template <int DT, int D, int N>
constexpr int smem_bytes() {
  using S = Shape<DT, D, N>;
  return S::kOffSh + (int)sizeof(Shared<S::kSlots, N>) + 1024;
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A descriptor of rows of `wide` bytes (128 or 64, swizzled at that width), 8 rows after one another.
__device__ __forceinline__ uint64_t rows_desc(uint32_t addr, int wide) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)((8 * wide) >> 4) << 32) | (1ull << 46) |
         ((wide == 128 ? 2ull : 4ull) << 61);
}
// Columns of the warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
               ::"memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t c;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(c) : "f"(hi), "f"(lo));
  return c;
}
__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}
// Two fp16 as terms of e5m2, each the top byte of its half of a word; the last one of three is rounded.
template <int TERMS, bool ROUND>
__device__ __forceinline__ void terms_of(uint32_t h, uint32_t (&w)[TERMS]) {
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    if (i + 1 == TERMS) {
      w[i] = ROUND && TERMS == 3 ? h + 0x00800080u : h;
    } else {
      w[i] = h & 0xff00ff00u;
      h = sub_half2(h, w[i]);
    }
  }
}
// The threads of warps 0-7 meet, each warp together; those of one half of the row-heads; the same and whether one of
// them says so.
__device__ __forceinline__ void sync_all() {
  __syncwarp();
  asm volatile("bar.sync 1, 256;" ::: "memory");
}
__device__ __forceinline__ void sync_half(int half) {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"r"(2 + half) : "memory");
}
__device__ __forceinline__ bool any_of_half(int half, bool p) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(4 + half)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(min(max(b, 95u), 158u) << 23); }   // 2^-32 .. 2^31

// A request's work: rows, tiles of N row-heads and steps, [c_lo, c_hi) of 128 tokens (one at least, if only to say 0).
struct Request {
  int64_t row0;
  int n, kv, total, tiles, c_lo, chunks;
  __device__ __forceinline__ int64_t weight(int Hkv) const { return (int64_t)Hkv * tiles * max(chunks, 1); }
};
template <int N>
__device__ __forceinline__ Request request_of(const ByteAttendArgs &a, int64_t r, bool report) {
  Request q = {};
  const int64_t row0 = a.row_off[r], row1 = a.row_off[r + 1], kv = a.kv_len[r], n = row1 - row0;
  int wrong = 0;
  if (row0 < 0 || n < 0 || row1 > a.rows) wrong = DSPARK_ERR_OFFSETS;
  else if (kv < 0 || kv > a.max_pages * a.page_size || n > a.max_rows) wrong = DSPARK_ERR_LENGTHS;
  if (wrong) {
    if (report) set_status(a.dev_status, wrong);
    return q;
  }
  q.row0 = row0, q.n = (int)n, q.kv = (int)kv, q.total = (int)n * a.group;
  q.tiles = (q.total + N - 1) / N;
  const int hi = a.causal ? q.kv - q.n + 1 : q.kv, lo = a.window ? max(hi, a.window) - a.window : 0;
  q.c_lo = lo / kTokens;
  q.chunks = max((q.kv + kTokens - 1) / kTokens - q.c_lo, 0);
  return q;
}

// A CTA's pieces, one after the other; every role walks them by itself.
template <int N>
struct Walk {
  int64_t r, at, left;           // request, place in its steps, steps to go
  Request q;
  int h, tile, ca, cb;           // the piece: head, tile, steps [ca, cb)
  bool begins, ends;             // whether it is its unit's first, its last
  __device__ __forceinline__ void start(const ByteAttendArgs &a, int64_t request, int64_t begin, int64_t steps) {
    r = request, at = begin, left = steps;
    if (left > 0) q = request_of<N>(a, r, false);
  }
  __device__ __forceinline__ bool next(const ByteAttendArgs &a) {
    if (left <= 0) return false;
    while (at >= q.weight(a.Hkv)) {
      at -= q.weight(a.Hkv);
      if (++r >= a.B) return false;
      q = request_of<N>(a, r, false);
    }
    const int each = max(q.chunks, 1);
    const int64_t unit = at / each;
    const int from = (int)(at - unit * each), steps = (int)min((int64_t)(each - from), left);
    h = (int)(unit / q.tiles), tile = (int)(unit - (int64_t)h * q.tiles);
    begins = from == 0, ends = from + steps == each;
    ca = q.c_lo + from, cb = q.c_lo + from + min(steps, q.chunks);
    at += steps, left -= steps;
    return true;
  }
};

template <int DT, int D, int N>
__global__ void __launch_bounds__(kThreads, Shape<DT, D, N>::kCtas)
    byte_attend_kernel(const __grid_constant__ ByteAttendArgs a, int run) {
  using T = typename Elem<DT>::T;
  using Sh = Shape<DT, D, N>;
  constexpr int kSlots = Sh::kSlots, kTerms = Sh::kTerms;
  // fp32 sums of e4m3 by e5m2; keys K-major (M = tokens), values MN-major (M = dimensions), queries and P K-major
  constexpr uint32_t kIdescS = (1u << 4) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kTokens >> 4) << 24);
  constexpr uint32_t kIdescO = (1u << 4) | (1u << 10) | (1u << 15) | ((uint32_t)(kTerms * N >> 3) << 17) | ((uint32_t)(D >> 4) << 24);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sb = (raw + 1023u) & ~1023u;
  uint8_t *gb = smem_raw + (sb - raw);
  auto &sh = *reinterpret_cast<Shared<kSlots, N> *>(gb + Sh::kOffSh);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int *abort = &sh.abort;
  grid_dep_launch();
  grid_dep_wait();
  if (tid == 0) {
    sh.abort = sh.odd = 0;
    sh.skip = read_status(a.dev_status);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    mbar_init(smem_u32(&sh.s_full[0]), 1);
    mbar_init(smem_u32(&sh.s_full[1]), 1);
    mbar_init(smem_u32(&sh.p_full), 8);
    mbar_init(smem_u32(&sh.o_done), 1);
    mbar_init(smem_u32(&sh.q_ready), 8);
    mbar_init(smem_u32(&sh.drain), 1);
    fence_barrier_init();
    sh.begin_request = -1;
  }
  // the steps of all requests before this thread's share of them
  const int64_t share = (a.B + kThreads - 1) / kThreads, r_lo = min(tid * share, a.B), r_hi = min(r_lo + share, a.B);
  int64_t mine = 0;
  for (int64_t r = r_lo; r < r_hi; ++r) mine += request_of<N>(a, r, blockIdx.x == 0).weight(a.Hkv);
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) sh.scan[warp] = upto;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) upto += total;
    total += sh.scan[w];
  }
  const int64_t ctas = min((int64_t)gridDim.x, total), k = blockIdx.x;
  const int64_t from = k < ctas ? total * k / ctas : 0, to = k < ctas ? total * (k + 1) / ctas : 0;
  if (k < ctas && from >= upto - mine && from < upto) {
    int64_t r = r_lo, at = from - (upto - mine);
    for (;; ++r) {
      const int64_t w = request_of<N>(a, r, false).weight(a.Hkv);
      if (at < w) break;
      at -= w;
    }
    sh.begin_request = r, sh.begin_at = at;
  }
  __syncthreads();
  if (sh.skip || sh.begin_request < 0) {
    if (tid == 0) a.headers[k] = make_int4(-1, 0, 0, 0);
    return;
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&sh.tmem), Sh::kAlloc);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem, o_tmem = tmem + 2 * N;
  const uint32_t full = smem_u32(sh.full), empty = smem_u32(sh.empty);
  Walk<N> walk;
  walk.start(a, sh.begin_request, sh.begin_at, to - from);

  if (warp == 8) {
    // ---------------- keys and values: K of the first step, then K of the next and V of each ----------------
    int idx = 0;
    bool ok = true;
    const int per = kTokens / run;
    while (ok && walk.next(a)) {
      if (walk.ca >= walk.cb) continue;
      const int32_t *table = a.table + walk.r * a.max_pages;
      const int hi = walk.q.kv, lo_hi = a.causal ? walk.q.kv - walk.q.n + 1 : walk.q.kv;
      const int lo = a.window ? max(lo_hi, a.window) - a.window : 0;
      // the lane's tokens of a step: `run` of one page, if a row may see one of them
      auto look_up = [&](int c) -> int32_t {
        const int t = c * kTokens + lane * run;
        return lane < per && c < walk.cb && t < hi && t + run > lo ? table[t / a.page_size] : -2;
      };
      auto bring = [&](int kind, int c, int32_t page) {
        const int s = idx % kSlots;
        const bool free = mbar_wait(empty + 8 * s, (uint32_t)(idx / kSlots & 1) ^ 1u, abort);
        if (!__all_sync(0xffffffffu, free)) return false;
        const int t = c * kTokens + lane * run;
        if (page < 0 ? page != -2 : page >= a.pages) {
          set_status(a.dev_status, DSPARK_ERR_PAGES);
          page = -2;
        }
        const uint32_t bytes = page >= 0 ? (uint32_t)(min(run, (hi - t + 15) / 16 * 16) * D) : 0u;
        const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0) mbar_arrive_tx(full + 8 * s, all);
        __syncwarp();
        if (bytes)
          bulk_g2s(sb + s * Sh::kSlot + lane * run * D,
                   a.data + ((((int64_t)page * a.Hkv + walk.h) * 2 + kind) * a.page_size + t % a.page_size) * D, bytes, full + 8 * s,
                   policy_evict_first());
        __syncwarp();
        ++idx;
        return true;
      };
      int32_t page = look_up(walk.ca), next = look_up(walk.ca + 1);
      ok = bring(0, walk.ca, page);
      for (int c = walk.ca; ok && c < walk.cb; ++c) {
        if (c + 1 < walk.cb) ok = bring(0, c + 1, next);
        const int32_t after = look_up(c + 2);
        if (ok) ok = bring(1, c, page);
        page = next, next = after;
      }
    }
    if (!ok && lane == 0)                                        // no copy may be under way at the end
      for (int i = max(idx - kSlots, 0); i < idx; ++i) {
        const long long begun = clock64();
        while (!mbar_try(full + 8 * (i % kSlots), (uint32_t)(i / kSlots & 1)) && clock64() - begun < kTimeoutCycles / 8) {
        }
      }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------- products ----------------
    // (the whole warp waits, one lane issues)
    int idx = 0, step = 0, piece = 0;
    bool ok = true;
    auto wait = [&](uint64_t &bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_try(smem_u32(&bar), parity) || mbar_wait(smem_u32(&bar), parity, abort)) != 0;
    };
    const uint64_t slots = rows_desc(sb, D), p_desc = rows_desc(sb + Sh::kOffP, 128), q_desc = rows_desc(sb + Sh::kOffQ, D);
    while (ok && walk.next(a)) {
      if (walk.ca >= walk.cb) continue;
      ok = wait(sh.q_ready, (uint32_t)(piece++ & 1));
      auto scores = [&](int s_no) {                              // of the keys in the next slot
        const int s = idx % kSlots;
        if (!wait(sh.full[s], (uint32_t)(idx / kSlots & 1))) return false;
        tc_fence_after();
        const uint64_t k_at = desc_on(slots, s * Sh::kSlot);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kTerms; ++i)
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
              mma_f8(tmem + (s_no & 1) * N, desc_on(k_at, x * 32), desc_on(q_desc, i * N * D + x * 32), kIdescS, i + x > 0);
          mma_commit(smem_u32(&sh.s_full[s_no & 1]));
          mma_commit(empty + 8 * s);
        }
        __syncwarp();
        ++idx;
        return true;
      };
      if (ok) ok = scores(step);
      for (int c = walk.ca; ok && c < walk.cb; ++c, ++step) {
        if (c + 1 < walk.cb) ok = scores(step + 1);
        if (ok) ok = wait(sh.p_full, (uint32_t)(step & 1));
        const int s = idx % kSlots;
        if (ok) ok = wait(sh.full[s], (uint32_t)(idx / kSlots & 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t v_at = desc_on(slots, s * Sh::kSlot);
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < kTokens / 32; ++x)
            mma_f8(o_tmem, desc_on(v_at, x * 32 * D), desc_on(p_desc, x * 32), kIdescO, c > walk.ca || x > 0);
          mma_commit(empty + 8 * s);
          mma_commit(smem_u32(&sh.o_done));
        }
        __syncwarp();
        ++idx;
      }
    }
    if (!ok && lane == 0) {
      set_status(a.dev_status, DSPARK_ERR_DEVICE_TIMEOUT);
      mma_commit(smem_u32(&sh.drain));
      const long long begun = clock64();
      while (!mbar_try(smem_u32(&sh.drain), 0) && clock64() - begun < kTimeoutCycles / 8) {
      }
    }
    __syncwarp();
  } else {
    // ---------------- scores to probabilities, sums to outputs ----------------
    // Row-heads are dealt to the halves in groups of 8, so that those of a tile that is not full leave work to both.
    constexpr int NG = N / 16, NC = 8 * NG;                      // groups and row-heads of a half
    const int half = warp >> 2, quad = warp & 3, t = tid & 127;
    auto col_of = [&](int g) { return 8 * (2 * g + half); };     // the first row-head of group g
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int dim = D == 128 ? t : quad * 16 + lane;             // of O^T: with 64 dimensions 16 lanes of each warp
    const bool has_dim = D == 128 || lane < 16;
    const uint32_t p_at = sb + Sh::kOffP;
    int step = 0, idx = 0;
    bool alive = true;                                           // a wait gave up: what follows keeps pace, with no result
    int4 header = make_int4(-1, 0, 0, 0);
    while (walk.next(a)) {
      const Request &q = walk.q;
      const int first = walk.tile * N, real = min(N, q.total - first), ctx = q.kv - q.n;
      const int hi_min = a.causal ? ctx + first / a.group + 1 : q.kv;
      const int hi_max = a.causal ? ctx + (first + real - 1) / a.group + 1 : q.kv;
      const int lo_min = a.window ? max(hi_min, a.window) - a.window : 0, lo_max = a.window ? max(hi_max, a.window) - a.window : 0;
      sync_all();                                                // (the last piece's sums have been read)
      // queries: 128 / N threads a row-head
      if (half == 0) {
        constexpr int kEach = 128 / N, kPieces = D / kEach / 8;
        const int c = tid / kEach, part = tid % kEach, rho = first + c;
        float x[kPieces * 8];
        float top = 0.0f;
        if (c < real) {
          const int tok = rho / a.group;
          const T *p = reinterpret_cast<const T *>(a.q) + (q.row0 + tok) * a.q_row +
                       (int64_t)(walk.h * a.group + rho - tok * a.group) * a.q_head + part * (kPieces * 8);
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const Eight<DT> v = reinterpret_cast<const Eight<DT> *>(p)[i];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[8 * i + j] = Elem<DT>::to(v.e[j]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kPieces * 8; ++i) x[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kPieces * 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
        for (int m = kEach / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        // by a power of two to below 2^15; rows of zeros and of infinities stay as they are
        const int e = (int)(__float_as_uint(top) >> 23);
        const int up = e == 0 || e == 255 ? 0 : min(127 + 14 - e, 126);
        const float f = copysignf(ldexpf(1.0f, up), a.scale_log2);  // the scale's sign goes with the queries
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          uint32_t w[4][kTerms];
#pragma unroll
          for (int j = 0; j < 4; ++j) terms_of<kTerms, false>(pack_half2(x[8 * i + 2 * j] * f, x[8 * i + 2 * j + 1] * f), w[j]);
          const int d = part * (kPieces * 8) + 8 * i, piece = d / 16;
          const int at = c * D + (D == 128 ? piece ^ (c & 7) : piece ^ ((c >> 1) & 3)) * 16 + d % 16;
#pragma unroll
          for (int k2 = 0; k2 < kTerms; ++k2)
            *reinterpret_cast<uint2 *>(gb + Sh::kOffQ + k2 * N * D + at) =
                make_uint2(__byte_perm(w[0][k2], w[1][k2], 0x7531), __byte_perm(w[2][k2], w[3][k2], 0x7531));
        }
        if (part == 0) {
          sh.R[c] = c < real ? fmaxf(ldexpf(fabsf(a.scale_log2), -up), 1e-37f) : 1.0f;
          sh.z[c] = c < real ? kNone : -INFINITY;
          sh.ref[c] = -INFINITY;
          sh.hi[c] = c < real ? (a.causal ? ctx + rho / a.group + 1 : q.kv) : 0;
        }
        if (tid == 0) sh.odd = 0;
      }
      fence_proxy_async_smem();
      sync_all();
      const bool some = walk.ca < walk.cb;
      const int mine = (real + 7) / 8 > half ? ((real + 7) / 8 - half + 1) / 2 : 0;   // groups with row-heads
      if (some && lane == 0) mbar_arrive(smem_u32(&sh.q_ready));
      __syncwarp();
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.0f;

      // The scales of the thread's token, a step ahead, and its page, two.  Its place (page of the text, token of the
      // page) moves on by the same numbers every step.
      const int32_t *table = a.table + walk.r * a.max_pages;
      const int blocks = a.page_size / kTileTokens, pages_on = kTokens / a.page_size, tokens_on = kTokens - pages_on * a.page_size;
      int at_page = (walk.ca * kTokens + t) / a.page_size, in_page = walk.ca * kTokens + t - at_page * a.page_size, at = walk.ca * kTokens + t;
      int32_t page = -1;
      int block = 0;
      auto look_up = [&]() {                                     // page and block of the token `at`; on to the next step's
        page = at < walk.cb * kTokens && at >= lo_min && at < hi_max ? table[at_page] : -1;
        block = in_page / kTileTokens;
        at += kTokens, at_page += pages_on, in_page += tokens_on;
        if (in_page >= a.page_size) in_page -= a.page_size, ++at_page;
      };
      uint32_t ks = 127, vs = 127;
      auto load_scales = [&]() {
        ks = vs = 127;
        if (page >= 0 && page < a.pages) {
          const uint8_t *s = a.scales + ((int64_t)page * a.Hkv + walk.h) * 2 * blocks + block;
          ks = s[0], vs = s[blocks];
        }
      };
      look_up();
      load_scales();
      look_up();
      // where V of a step lies in the ring: K0, K1, V0, K2, V1, ...
      for (int c = walk.ca; c < walk.cb; ++c, ++step) {
        const bool at_first = c == walk.ca;
        const int v_idx = idx + (c + 1 < walk.cb ? (at_first ? 2 : 1) : (at_first ? 1 : 0));
        idx = v_idx + 1;
        const float A = scale_of(ks), w = scale_of(vs), lw = (float)((int)min(max(vs, 95u), 158u) - 127);
        load_scales();
        look_up();
        const int base = c * kTokens, tok = base + t;
        const bool edge = base < lo_max || base + kTokens > hi_min;
        const bool mine_ok = mbar_try(smem_u32(&sh.s_full[step & 1]), (uint32_t)(step >> 1 & 1)) ||
                             mbar_wait(smem_u32(&sh.s_full[step & 1]), (uint32_t)(step >> 1 & 1), abort);
        alive = __all_sync(0xffffffffu, mine_ok) && alive;
        tc_fence_after();
        // `G` groups of row-heads (what P holds of others, past the last, reaches no output)
        auto scores_to_terms = [&](auto groups) {
          constexpr int G = decltype(groups)::value;
          unsigned long long y[4 * G];
          auto load_scores = [&]() {                             // the token's scores, scaled and masked
            const unsigned long long A2 = f2_pack(A, A);
            uint32_t s[G][8];
#pragma unroll
            for (int g = 0; g < G; ++g) tmem_ld(tmem + lanes + (step & 1) * N + col_of(g), s[g]);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              tmem_wait(s[g]);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                y[g * 4 + j] = f2_mul(f2_pack(__uint_as_float(s[g][2 * j]), __uint_as_float(s[g][2 * j + 1])), A2);
            }
            if (edge) {
#pragma unroll
              for (int j = 0; j < 4 * G; ++j) {
                float y0, y1;
                f2_unpack(y[j], y0, y1);
                const int h0 = sh.hi[col_of(j / 4) + 2 * (j & 3)], h1 = sh.hi[col_of(j / 4) + 2 * (j & 3) + 1];
                if (!(tok < h0 && (!a.window || tok >= h0 - a.window))) y0 = -INFINITY;
                if (!(tok < h1 && (!a.window || tok >= h1 - a.window))) y1 = -INFINITY;
                y[j] = f2_pack(y0, y1);
              }
              __syncwarp();
            }
          };
          auto exponents = [&]() {                               // of their probabilities, in their place, and the largest
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2 * G; ++j) {
              const int c2 = col_of(j / 2) + 4 * (j & 1);
              const ulonglong2 r2 = *reinterpret_cast<const ulonglong2 *>(sh.R + c2), z2 = *reinterpret_cast<const ulonglong2 *>(sh.z + c2);
              float x0, x1, x2, x3;
              y[2 * j] = f2_fma(y[2 * j], r2.x, z2.x);
              y[2 * j + 1] = f2_fma(y[2 * j + 1], r2.y, z2.y);
              f2_unpack(y[2 * j], x0, x1);
              f2_unpack(y[2 * j + 1], x2, x3);
              most = fmaxf(fmaxf(most, fmaxf(x0, x1)), fmaxf(x2, x3));
            }
            return most;
          };
          // (one copy of the code whether a reference moves or not: what was loaded is loaded again then)
          for (int round = 0;; ++round) {
            load_scores();
            if (round != 1) {
              const float most = exponents();
              if (round == 2 || !any_of_half(half, most + lw > kBar)) break;
              continue;
            }
            // references move
#pragma unroll
            for (int j = 0; j < 4 * G; ++j) {
              const int c2 = col_of(j / 4) + 2 * (j & 3);
              float y0, y1;
              f2_unpack(y[j], y0, y1);
              float m2[2] = {fmaf(y0, sh.R[c2], lw), fmaf(y1, sh.R[c2 + 1], lw)};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float x = m2[i] == m2[i] ? m2[i] : -INFINITY;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                if (lane == 0) sh.most[quad][c2 + i] = x;
              }
            }
            sync_half(half);
            if (t < 8 * G) {
              const int c2 = col_of(t >> 3) + (t & 7);
              const float was = sh.ref[c2];
              const float up = fmaxf(fmaxf(fmaxf(sh.most[0][c2], sh.most[1][c2]), fmaxf(sh.most[2][c2], sh.most[3][c2])), was);
              sh.factor[c2] = was == -INFINITY ? 0.0f : fast_ex2(was - up);
              sh.ref[c2] = up;
              if (up != -INFINITY && c2 < real) sh.z[c2] = kTop - up;
            }
            sync_half(half);
#pragma unroll
            for (int c = 0; c < 8 * G; ++c) l[c] *= sh.factor[col_of(c >> 3) + (c & 7)];
            if (!at_first) {
              const bool done = mbar_try(smem_u32(&sh.o_done), (uint32_t)((step - 1) & 1)) ||
                              mbar_wait(smem_u32(&sh.o_done), (uint32_t)((step - 1) & 1), abort);
              alive = __all_sync(0xffffffffu, done) && alive;
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < kTerms; ++i)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                  const uint32_t o_at = o_tmem + lanes + i * N + col_of(g);
                  uint32_t o[8];
                  tmem_ld(o_at, o);
                  tmem_wait(o);
#pragma unroll
                  for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sh.factor[col_of(g) + j]);
                  tmem_st(o_at, o);
                }
              tmem_wait_st();
              tc_fence_before();
            }
          }
          // probabilities in terms; the place of a byte in P: a row of 128, its 16-byte piece swizzled by the row
          if (!at_first) {
            const bool done = mbar_try(smem_u32(&sh.o_done), (uint32_t)((step - 1) & 1)) ||
                              mbar_wait(smem_u32(&sh.o_done), (uint32_t)((step - 1) & 1), abort);
            alive = __all_sync(0xffffffffu, done) && alive;
          }
          const unsigned long long w2 = f2_pack(w, w);
          const uint32_t p_col = p_at + 8 * half * kTokens;
#pragma unroll
          for (int j = 0; j < 4 * G; ++j) {
            constexpr int kGap = 16 * kTokens;
            float x0, x1;
            f2_unpack(y[j], x0, x1);
            const float p0 = fast_ex2(x0), p1 = fast_ex2(x1);
            l[2 * j] += p0;
            l[2 * j + 1] += p1;
            float v0, v1;
            f2_unpack(f2_mul(f2_pack(p0, p1), w2), v0, v1);
            uint32_t x[kTerms];
            terms_of<kTerms, true>(pack_half2(v0, v1), x);
            const uint32_t to0 = p_col + (t ^ ((2 * j & 7) << 4)) + j / 4 * kGap + 2 * (j & 3) * kTokens;
            const uint32_t to1 = p_col + (t ^ (((2 * j + 1) & 7) << 4)) + j / 4 * kGap + (2 * (j & 3) + 1) * kTokens;
#pragma unroll
            for (int i = 0; i < kTerms; ++i) {
              asm volatile("st.shared.u8 [%0], %1;" ::"r"(to0 + i * N * kTokens), "r"(x[i] >> 8) : "memory");
              asm volatile("st.shared.u8 [%0], %1;" ::"r"(to1 + i * N * kTokens), "r"(x[i] >> 24) : "memory");
            }
          }
        };
        if (NG >= 4 && mine > 2)
          scores_to_terms(std::integral_constant<int, NG>());
        else if (NG >= 2 && mine > 1)
          scores_to_terms(std::integral_constant<int, NG < 2 ? NG : 2>());
        else if (mine > 0)
          scores_to_terms(std::integral_constant<int, 1>());
        else if (!at_first) {                                    // no row-head here: this half keeps pace
          const bool done = mbar_try(smem_u32(&sh.o_done), (uint32_t)((step - 1) & 1)) ||
                            mbar_wait(smem_u32(&sh.o_done), (uint32_t)((step - 1) & 1), abort);
          alive = __all_sync(0xffffffffu, done) && alive;
        }
        if (edge) {
          // A value of a token that no row of the tile sees is whatever the page held, one that some rows do not see
          // may be a NaN, and 0 NaN would reach them: both leave the product.  (All uses of the ring before this
          // step's are done, so the phase waited for is this one.)
          const int s = v_idx % kSlots;
          const bool there = mbar_wait(full + 8 * s, (uint32_t)(v_idx / kSlots & 1), abort);
          alive = __all_sync(0xffffffffu, there) && alive;
          uint4 *v = reinterpret_cast<uint4 *>(gb + s * Sh::kSlot + t * D) + half * (D / 32);   // half of the value each
          const bool seen = tok >= lo_min && tok < hi_max;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint4 x = v[i];
            if (!seen) {
              v[i] = make_uint4(0, 0, 0, 0);
            } else {
              uint32_t *e = reinterpret_cast<uint32_t *>(&x);
              uint32_t found = 0;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t nan = ((e[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                e[j] &= ~((nan >> 7) * 0xffu);
                found |= nan;
              }
              if (found) {
                v[i] = x;
                sh.odd = 1;
              }
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full));
        __syncwarp();
      }

      // ---------------- the piece's sums ----------------
      if (some) {
        const bool done = mbar_try(smem_u32(&sh.o_done), (uint32_t)((step - 1) & 1)) ||
                            mbar_wait(smem_u32(&sh.o_done), (uint32_t)((step - 1) & 1), abort);
        alive = __all_sync(0xffffffffu, done) && alive;
        tc_fence_after();
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (col_of(c >> 3) >= real) break;
        float x = l[c];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (lane == 0) sh.sum[quad][col_of(c >> 3) + (c & 7)] = x;
      }
      sync_all();
      const bool whole = walk.begins && walk.ends, odd = *(volatile int *)&sh.odd != 0;
      float *partial = a.partial + (2 * k + (walk.begins ? 1 : 0)) * Sh::kPartial;
      if (!whole && tid < N) {
        partial[tid] = sh.ref[tid];
        partial[N + tid] = sh.sum[0][tid] + sh.sum[1][tid] + sh.sum[2][tid] + sh.sum[3][tid];
      }
      __syncwarp();
#pragma unroll 1
      for (int g = 0; g < NG; ++g) {
        const int c0 = col_of(g);
        if (c0 >= real) break;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
        if (some) {
#pragma unroll
          for (int i = 0; i < kTerms; ++i) {
            uint32_t o[8];
            tmem_ld(o_tmem + lanes + i * N + c0, o);
            tmem_wait(o);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += __uint_as_float(o[j]);
          }
        }
        if (odd && has_dim)
          for (int c = walk.ca; c < walk.cb; ++c) {
            if (!(c * kTokens < lo_max || c * kTokens + kTokens > hi_min)) continue;
            for (int x = max(c * kTokens, lo_min); x < min(c * kTokens + kTokens, hi_max); ++x) {
              const int32_t pg = table[x / a.page_size];
              if (pg < 0 || pg >= a.pages) continue;
              const int in = x % a.page_size, piece = D == 128 ? (dim / 16) ^ (in & 7) : (dim / 16) ^ ((in >> 1) & 3);
              const uint8_t held = a.data[((((int64_t)pg * a.Hkv + walk.h) * 2 + 1) * a.page_size + in) * D + piece * 16 + dim % 16];
              if ((held & 0x7f) != 0x7f) continue;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int hi = sh.hi[c0 + j];
                if (x < hi && (!a.window || x >= hi - a.window)) y[j] = __int_as_float(0x7fffffff);
              }
            }
          }
        __syncwarp();
        if (alive && has_dim) {
          int tok = (first + c0) / a.group, sub = first + c0 - tok * a.group;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = c0 + j;
            if (c >= real) break;
            if (whole) {
              const float sum = sh.sum[0][c] + sh.sum[1][c] + sh.sum[2][c] + sh.sum[3][c];
              const int64_t at = (q.row0 + tok) * a.Hq + walk.h * a.group + sub;
              reinterpret_cast<T *>(a.out)[at * D + dim] = Elem<DT>::from(sum == 0.0f ? 0.0f : y[j] / sum);
              if (a.lse && dim == 0)
                a.lse[at] = sum == 0.0f ? -INFINITY : kLn2 * (sh.ref[c] == -INFINITY ? 0.0f : sh.ref[c] - kTop) + logf(sum);
            } else {
              partial[2 * N + c * D + dim] = y[j];
            }
            if (++sub == a.group) sub = 0, ++tok;
          }
        }
        __syncwarp();
      }
      if (!whole && walk.begins) {
        // the unit goes on in the CTAs up to the one that has its last step; this is the CTA's last piece
        const int64_t last = to - 1 + max(walk.q.chunks, 1) - (walk.cb - walk.ca);
        const int64_t until = ((last + 1) * ctas - 1) / total;
        header = make_int4((int)walk.r, walk.h, walk.tile, (int)(until - k + 1));
      }
    }
    if (tid == 0) a.headers[k] = header;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, Sh::kAlloc);
}

// Joins the pieces of the unit that began in CTA blockIdx.x / groups and went on: a warp takes a row-head.
template <int DT, int D, int N>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ ByteAttendArgs a) {
  using T = typename Elem<DT>::T;
  using Sh = Shape<DT, D, N>;
  constexpr int kGroups = N / 4, kMine = D / 32;
  const int lane = threadIdx.x & 31, c = (int)(blockIdx.x % kGroups) * 4 + (threadIdx.x >> 5);
  const int64_t k = blockIdx.x / kGroups;
  grid_dep_launch();
  grid_dep_wait();
  if (read_status(a.dev_status)) return;
  const int4 head = a.headers[k];
  if (head.x < 0) return;
  const int64_t row0 = a.row_off[head.x], n = a.row_off[head.x + 1] - row0;
  const int rho = head.z * N + c, parts = head.w;
  if (rho >= n * a.group) return;
  // the first piece is slot 1 of CTA k, the others slot 0 of those after it
  auto slot = [&](int p) { return a.partial + (p ? 2 * (k + p) : 2 * k + 1) * Sh::kPartial; };
  float big = -INFINITY;
  for (int p = lane; p < parts; p += 32) big = fmaxf(big, slot(p)[c]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
  float sum = 0.0f, y[kMine] = {};
  for (int p0 = 0; p0 < parts; p0 += 32) {
    float f = 0.0f;
    if (p0 + lane < parts) {
      const float *s = slot(p0 + lane);
      const float m = s[c], l = s[N + c];
      // (a piece whose every score was a NaN has no reference but a sum)
      f = l == 0.0f ? 0.0f : (m == -INFINITY || big == -INFINITY ? 1.0f : fast_ex2(m - big));
      sum = fmaf(l, f, sum);
    }
    const int here = min(32, parts - p0);
    for (int p1 = 0; p1 < here; p1 += 8) {                        // 8 pieces' rows under way
      float2 u[8][kMine / 2];
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p1 + p < here)
#pragma unroll
          for (int i = 0; i < kMine / 2; ++i)
            u[p][i] = reinterpret_cast<const float2 *>(slot(p0 + p1 + p) + 2 * N + c * D + lane * kMine)[i];
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float g = __shfl_sync(0xffffffffu, f, (p1 + p) & 31);
        if (p1 + p < here && g != 0.0f)
#pragma unroll
          for (int i = 0; i < kMine / 2; ++i) {
            y[2 * i] = fmaf(u[p][i].x, g, y[2 * i]);
            y[2 * i + 1] = fmaf(u[p][i].y, g, y[2 * i + 1]);
          }
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = (row0 + rho / a.group) * a.Hq + head.y * a.group + rho % a.group;
  T *to = reinterpret_cast<T *>(a.out) + at * D + lane * kMine;
#pragma unroll
  for (int i = 0; i < kMine; ++i) to[i] = Elem<DT>::from(y[i] * inv);
  if (a.lse && lane == 0) a.lse[at] = sum == 0.0f ? -INFINITY : kLn2 * (big == -INFINITY ? 0.0f : big - kTop) + logf(sum);
}

// Row-heads of a tile: what the largest request has, up to 64.
int tile_of(int64_t row_heads) { return row_heads <= 16 ? 16 : (row_heads <= 32 ? 32 : 64); }
int64_t grid_of(int n, int sms) { return (n <= 32 ? 2 : 1) * (int64_t)sms; }

template <int DT, int D, int N>
cudaError_t launch(const ByteAttendArgs &a, cudaStream_t s, int sms) {
  auto *fn = byte_attend_kernel<DT, D, N>;
  constexpr int smem = smem_bytes<DT, D, N>();
  cudaError_t e = ensure_dynamic_smem((const void *)fn, smem);
  if (e != cudaSuccess) return e;
  int run = 16;                                                   // tokens of a step that lie in one page
  while (run < kTokens && a.page_size % (2 * run) == 0) run *= 2;
  const int64_t grid = grid_of(N, sms);
  e = launch_next(fn, grid, kThreads, smem, 1, s, a, run);
  return e != cudaSuccess ? e : launch_next(join_kernel<DT, D, N>, grid * (N / 4), 128, 0, 1, s, a);
}
template <int DT, int D>
cudaError_t launch_rows(const ByteAttendArgs &a, cudaStream_t s, int sms) {
  const int n = tile_of((int64_t)a.max_rows * a.group);
  return n == 16 ? launch<DT, D, 16>(a, s, sms) : (n == 32 ? launch<DT, D, 32>(a, s, sms) : launch<DT, D, 64>(a, s, sms));
}

}  // namespace

// Two pieces' sums and a header for every CTA.
int64_t byte_attend_workspace_bytes(int group, int D, int64_t max_rows, int sms) {
  const int n = tile_of(max_rows * group);
  return grid_of(n, sms) * (2 * (int64_t)n * (D + 2) * 4 + (int64_t)sizeof(int4));
}

cudaError_t launch_byte_attend(const ByteAttendArgs &args, void *workspace, cudaStream_t s, int sms) {
  ByteAttendArgs a = args;
  const int n = tile_of((int64_t)a.max_rows * a.group);
  a.headers = (int4 *)workspace;
  a.partial = (float *)(a.headers + grid_of(n, sms));
  if (a.dtype == DSPARK_BF16) return a.D == 128 ? launch_rows<DSPARK_BF16, 128>(a, s, sms) : launch_rows<DSPARK_BF16, 64>(a, s, sms);
  return a.D == 128 ? launch_rows<DSPARK_F16, 128>(a, s, sms) : launch_rows<DSPARK_F16, 64>(a, s, sms);
}

}  // namespace dspark
