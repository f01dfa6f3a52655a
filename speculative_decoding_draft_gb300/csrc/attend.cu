// Attention of ragged rows over a paged cache held in 4 bits.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - m),  lse = m + log sum_t p_t
// over the tokens t that a row sees: t < hi, hi = kv_len (causal: kv_len - n + j + 1 for row j of n),
// and t >= hi - window with a window.  A row that sees nothing gets 0 and lse = -inf.
//
// One pass over the cache.  A warp takes 32 tokens (64 of heads with 64 dimensions) at a time, brought by
// bulk copies into a ring of its own, and works transposed: S^T = K Q^T and O^T = V^T P^T with m16n8k16 products, so
// the tokens (then the dimensions) fill the 16-wide side and the 8-wide side holds the rows: the
// query heads of one key/value head times the request's rows, 8 for plain decoding with up to 8
// heads a group, with nothing padded to 16, 64 or 128.  The 4-bit operands go straight from shared
// memory into the registers of the product: the layout of a tile gives each thread its own bytes, a
// hardware conversion makes two fp16 of a byte and one multiplication by the scale makes the exact
// element.  Both inner orders are free (the dimensions of q.k, the dimensions of the output), which
// is what lets a thread take neighbouring bytes.  P^T is turned into the second product's operand
// with one matrix transposition in registers per 8x8.
//
// Rounding: queries are scaled by a power of two to below 2^9 and rounded to fp16 (exact for bf16 and
// fp16 queries down to 2^-33 of the row's largest), keys and values are exact, probabilities are
// rounded to fp16 (2^-12), everything else and all sums are fp32.
//
// The running maximum moves only when a score passes it by 2^8: probabilities then lie below 2^14
// (they are kept 2^6 up so that small ones stay normal fp16 numbers), the result is the same, and the
// reductions over lanes and the rescaling of the output leave the common path.
//
// The tokens of one (request, key/value head, row tile) are dealt to the warps of a CTA, of a cluster of
// CTAs where there are too few units to fill the SMs, or of many CTAs that meet through a workspace where
// eight still are; partial results meet in shared memory, across the cluster, or in merge_kernel.  Requests
// start longest first.
//
// Measured (one GB300): 64 requests of 512 to 4096 tokens with 1 to 8 rows, 32 query and 8 key/value heads
// of 128 dimensions 76 us (26 us of reading at the memory's rate); one request of 131071 tokens with 8 rows
// 77 us (22); 256 requests of up to 16384 tokens, heads of 64 dimensions, 265 us (202).  Bound by the issue
// slots and what fills them: a warp's step of 32 tokens by 16 rows is about 700 instructions, 136 of them
// conversions and 128 scalings, both at half rate, and 64 products; the SMs issue 1.8 to 2.2 a cycle.
// Tried and slower or no faster for the 64 requests: 16 warps an SM with 35 words spilled a step (85 us), 32
// rows a warp (90), 8 rows (104), two warps sharing a step of 32 rows with half of the output each (133), steps
// of 16 tokens (84) and of 64 (86), chunks drawn from a counter instead of dealt (no faster, and not
// reproducible).  The fifth-generation tensor cores take operands from shared or tensor memory only, where
// every expanded element would have to be written and read again: 512 bytes a token and head each way (fp16, 128
// dimensions) against the 144 that are stored.  At the memory's rate an SM receives 23 stored bytes a cycle, so
// that is 83 bytes in and 83 out of shared memory's 128 a cycle: 1.3 times what it can move meanwhile, or 34 us
// for the 64 requests if nothing else used it.  One expansion would then serve all row-heads of a key/value head,
// which pays where there are many (prompts, whose tiles of 16 or 32 rows each expand the cache again).  Not built.
#include <type_traits>

#include <cooperative_groups.h>

#include "attn.cuh"

namespace dspark {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kStages = 2;            // of a warp's ring; three took 2 us more, shared memory that CTAs want
// CTAs on an SM together by the n-tiles of a warp: what their registers allow without spilling in the loop
// (16 rows at 4 CTAs spill 35 words a step: 85 us for the 64 requests against 76 at 3).
__host__ __device__ constexpr int ctas_of(int nt, int D) { return nt == 4 ? 2 : (nt == 1 && D == 64 ? 4 : 3); }
constexpr float kLazy = 8.0f;         // how far (log2) a score may pass the running maximum
constexpr float kLift = 6.0f;         // probabilities are kept 2^kLift up

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same on an accumulator of zeros.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The four bytes of a word, each two e2m1 codes, as four pairs of fp16.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 x, y, z, t;\n\t"
      "mov.b32 {x, y, z, t}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, x;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, y;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, z;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, t;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t e4m3x2(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(h) : "r"(two));
  return h;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t c;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(c) : "f"(hi), "f"(lo));
  return c;
}

// Plain loads: the compiler may move them among the products, but not over a wait.
template <int BYTES>
__device__ __forceinline__ void lds(const uint8_t *p, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES == 16) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x, w[1] = v.y;
  }
}
__device__ __forceinline__ uint32_t lds_u16(const uint8_t *p) { return *reinterpret_cast<const uint16_t *>(p); }
__device__ __forceinline__ uint32_t lds_u8(const uint8_t *p) { return *p; }

// The i-th request, long ones first: CTAs start in the order of their index, and one that starts last must
// not be the longest (64 requests 85 us, 97 in the order given; 256 requests 266, 300).  Eight classes by
// length; every warp works it out by itself from the lengths, as long as it can hold these (B <= 256).  More
// requests start in the order given, which costs less the more there are: of up to 4096 tokens with 1 to 8 rows
// 300 take 332 us (314 if given longest first) and 512 take 534 (515), 2048 of up to 2048 tokens 1308 (1293);
// with heads of 64 dimensions and 1 or 2 rows 512 of up to 16384 tokens take 505 (455).
constexpr int kOrderMost = 256;
__device__ __forceinline__ int64_t longest_first(const int32_t *kv_len, int64_t B, int64_t i, int lane) {
  if (B > kOrderMost || B < 2) return i;
  int len[kOrderMost / 32], most = 1;
#pragma unroll
  for (int j = 0; j < kOrderMost / 32; ++j) {
    len[j] = 32 * j + lane < B ? max(kv_len[32 * j + lane], 0) : -1;
    most = max(most, len[j]);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  const float scale = 7.999f / (float)most;
  int left = (int)i;
  for (int c = 7; c >= 0; --c) {
#pragma unroll
    for (int j = 0; j < kOrderMost / 32; ++j) {
      if (32 * j >= B) break;
      const uint32_t in = __ballot_sync(0xffffffffu, len[j] >= 0 && (int)((float)len[j] * scale) == c);
      const int n = __popc(in);
      if (left < n) return 32 * j + __fns(in, 0, left + 1);
      left -= n;
    }
  }
  return i;                                  // not reached
}

template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTiles = 256 / D;                           // tiles of a warp's step: 64 or 32 tokens
  static constexpr int kChunk = kTiles * kTileTokens;
  static constexpr int kStage = kTiles * tile_bytes(D);
  static constexpr int kRing = kStages * kStage;                    // per warp
  static constexpr int kOutRow = D + 4;                            // floats; padded against bank conflicts
  static constexpr int kOut = kRows * kOutRow * 4;                 // one warp's partial output
  static constexpr int kWarpBytes = (kRing > kOut ? kRing : kOut); // the ring is reused for it
  static constexpr bool kQShared = NT > 1;                         // query fragments stay in shared memory
  static constexpr int kQ = NT * (D / 16) * 32 * 8;
  static constexpr int kBars = kWarps * kStages * 8;
  static constexpr int kMl = kWarps * kRows * 8 + kRows * 12;      // maxima and sums of the warps, of the CTA; scales
  static constexpr int kPlaces = kWarps * kTiles * 16 + 48;        // the ring's places, see below
  static constexpr int kSmem = kWarps * kWarpBytes + kQ + kBars + kPlaces + kMl + 16;
  static constexpr int kPartial = kRows * (D + 2);                 // floats of a CTA's partial result
};

template <int DT, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, ctas_of(NT, D))
    attend_kernel(const __grid_constant__ AttendArgs a, int row_tiles, int parts) {
  using T = typename Elem<DT>::T;
  using Sh = Shape<D, NT>;
  constexpr int KS = D / 16;                 // k-steps of q.k, and m-tiles of the output
  constexpr int TC = Sh::kTiles, kChunk = Sh::kChunk;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *q_smem = smem + kWarps * Sh::kWarpBytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(q_smem + Sh::kQ);
  int4 *places = reinterpret_cast<int4 *>(bars + kWarps * kStages), *fixed = places + kWarps * TC;
  float *warp_m = reinterpret_cast<float *>(fixed + 3);
  float *warp_l = warp_m + kWarps * Sh::kRows;
  float *cta_m = warp_l + kWarps * Sh::kRows, *cta_l = cta_m + Sh::kRows;
  float *row_scale = cta_l + Sh::kRows;
  volatile int *abort = reinterpret_cast<volatile int *>(row_scale + Sh::kRows);

  cg::cluster_group cluster = cg::this_cluster();
  const int cs = (int)cluster.num_blocks(), rank = (int)(blockIdx.x % (unsigned)parts);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  grid_dep_launch();
  grid_dep_wait();
  int64_t unit = blockIdx.x / (unsigned)parts;
  const int rt = (int)(unit % row_tiles);
  unit /= row_tiles;
  const int h = (int)(unit % a.Hkv);
  const int64_t r = longest_first(a.kv_len, a.B, unit / a.Hkv, lane);
  const int64_t row0 = a.row_off[r], row1 = a.row_off[r + 1], kv = a.kv_len[r];
  const int64_t n = row1 - row0;
  // every CTA of a cluster takes the same way out here
  if (row0 < 0 || n < 0 || row1 > a.rows) {
    if (tid == 0) set_status(a.dev_status, DSPARK_ERR_OFFSETS);
    return;
  }
  if (kv < 0 || kv > a.max_pages * a.page_size || n > a.max_rows) {
    if (tid == 0) set_status(a.dev_status, DSPARK_ERR_LENGTHS);
    return;
  }
  const int first = rt * Sh::kRows, total = (int)n * a.group;
  if (first >= total) return;
  const int last = (first + Sh::kRows < total ? first + Sh::kRows : total) - 1;
  // a step that failed does no work, but its CTAs still meet their cluster below
  const bool skip = status_on_entry(a.dev_status) != 0;

  // what the tile's rows see: from [lo_min, lo_max] up to [hi_min, hi_max]
  const int ctx = (int)(kv - n);
  const int hi_min = a.causal ? ctx + first / a.group + 1 : (int)kv;
  const int hi_max = a.causal ? ctx + last / a.group + 1 : (int)kv;
  // (ends may be negative: what is subtracted from is the larger of end and window)
  const int lo_min = a.window ? max(hi_min, a.window) - a.window : 0;
  const int lo_max = a.window ? max(hi_max, a.window) - a.window : 0;
  const int c0 = lo_min / kChunk;
  const int chunks = skip || hi_max <= 0 ? 0 : (hi_max + kChunk - 1) / kChunk - c0;

  const uint32_t ring = smem_u32(smem) + warp * Sh::kWarpBytes;
  const uint32_t bar = smem_u32(bars + warp * kStages);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bar + 8 * i, 1);
    if (warp == 0) *abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();

  // The ring.  Where a step's tiles always lie in one page, lane 0 brings them with one copy, else one lane
  // each.  A lane's place (piece, page, piece in the page) moves on by the same numbers every step, so it
  // follows by an addition; the page's id is looked up a step ahead.  Places and numbers live in shared
  // memory: registers are what the loop below is short of.
  const int step = parts * kWarps, w0 = rank * kWarps + warp;
  const int32_t *table = a.table + r * a.max_pages;
  const int tiles_per_page = a.page_size / kTileTokens;
  int32_t page = -1;
  bool gone = false;
  {
    const bool whole = tiles_per_page % TC == 0;
    const int per_page = whole ? tiles_per_page / TC : tiles_per_page, per_step = whole ? 1 : TC;
    const int ahead = per_step * step, pieces = whole ? c0 + chunks : (hi_max + kTileTokens - 1) / kTileTokens;
    if (tid == 0) {
      fixed[0] = make_int4(ahead, ahead / per_page, ahead % per_page, per_page);
      fixed[1] = make_int4(whole ? TC * tile_bytes(D) : tile_bytes(D), pieces, h, chunks);
      fixed[2] = make_int4((int)row0, skip ? 0 : total, first, 0);      // no rows to store where the step had failed
    }
    if (lane < TC) {
      const int piece = lane < per_step ? per_step * (c0 + w0) + lane : 0x3fffffff;
      places[warp * TC + lane] = make_int4(piece, piece / per_page, piece % per_page, 0);
      // The first step may hold tiles that lie before the window altogether.  Their pages may be gone: they are not
      // looked up.
      gone = !whole && piece < lo_min / kTileTokens;
      if (w0 < chunks && !gone && piece < pieces) page = table[piece / per_page];
    }
    __syncthreads();
  }
  auto issue = [&](int c, int stage, bool gone) {       // chunk c, and the look-up for chunk c + step
    if (lane < TC) {
      constexpr uint32_t kLanes = (1u << TC) - 1;
      const int4 by = fixed[0], k = fixed[1];
      int4 at = places[warp * TC + lane];
      const bool want = at.x < k.y && !gone, ok = want && page >= 0 && page < a.pages;
      if (want && !ok) set_status(a.dev_status, DSPARK_ERR_PAGES);
      const uint32_t got = __ballot_sync(kLanes, ok);
      if (lane == 0) mbar_arrive_tx(bar + 8 * stage, __popc(got) * k.x);
      __syncwarp(kLanes);
      if (ok)
        bulk_g2s(ring + stage * Sh::kStage + lane * tile_bytes(D),
                 a.cache + ((int64_t)page * a.Hkv + k.z) * (tiles_per_page * tile_bytes(D)) + at.z * k.x, k.x,
                 bar + 8 * stage, policy_evict_first());
      at.x += by.x;
      at.y += by.y;
      at.z += by.z;
      if (at.z >= by.w) {
        at.z -= by.w;
        ++at.y;
      }
      places[warp * TC + lane] = at;
      page = c + step < k.w && at.x < k.y ? table[at.y] : -1;
    }
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i)
    if (w0 + i * step < chunks) issue(w0 + i * step, i, i == 0 && gone);

  // Queries, an n-tile a warp: a lane has row g, dimensions [q4 D/4, (q4 + 1) D/4).
  if (warp < NT) {
    const int rho = first + 8 * warp + g;
    float x[D / 4];
    float top = 0.0f;
    if (rho < total) {
      const T *p = reinterpret_cast<const T *>(a.q) + (row0 + rho / a.group) * a.q_row +
                   (int64_t)(h * a.group + rho % a.group) * a.q_head + q4 * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const Eight<DT> v = reinterpret_cast<const Eight<DT> *>(p)[i];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[8 * i + k] = Elem<DT>::to(v.e[k]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 4; ++i) x[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // by 2^(8 - e), e the exponent of the row's largest; rows of zeros and of infinities stay as they are
    const int e = (int)(__float_as_uint(top) >> 23);
    const int up = e == 0 || e == 255 ? 0 : min(127 + 8 - e, 126);
    const float f = copysignf(ldexpf(1.0f, up), a.scale_log2);   // the scale's sign goes with the queries,
    if (q4 == 0) row_scale[8 * warp + g] = fmaxf(ldexpf(fabsf(a.scale_log2), -up), 1e-37f);   // so that maxima can
#pragma unroll                                                                                // be taken unscaled
    for (int s = 0; s < KS; ++s)
      reinterpret_cast<uint2 *>(q_smem)[((warp * KS + s) / 2 * 32 + lane) * 2 + (s & 1)] =
          make_uint2(pack2(x[4 * s] * f, x[4 * s + 1] * f), pack2(x[4 * s + 2] * f, x[4 * s + 3] * f));
  }
  __syncthreads();
  uint32_t qf[Sh::kQShared ? 1 : KS / 2][4];
  if constexpr (!Sh::kQShared) {
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) lds<16>(q_smem + (i * 32 + lane) * 16, qf[i]);
  }
  // score of rows 2 q4 and 2 q4 + 1 = row_scale * accumulator, in log2; row_scale > 0
  const float2 *scales = reinterpret_cast<const float2 *>(row_scale) + q4;
  auto end_of = [&](int nt, int k) {         // where the tokens end that such a row sees
    const int rho = first + 8 * nt + 2 * q4 + k;
    return rho >= total ? 0 : (a.causal ? ctx + rho / a.group + 1 : (int)kv);
  };

  // Probabilities are 2^(score + z), z = kLift - the running maximum in log2, which moves when an
  // accumulator passes bar_at (-inf: no maximum yet, z = 0).
  float o[NT][KS][4], l[NT][2], z[NT][2] = {}, bar_at[NT][2] = {};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.0f;
    bar_at[nt][0] = bar_at[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = z[nt][0] = z[nt][1] = 0.0f;
  }

  auto maximum = [&](int nt, int k) { return bar_at[nt][k] == -INFINITY ? -INFINITY : kLift - z[nt][k]; };
  // One chunk: buf holds its tiles, base is its first token; an EDGE one holds tokens that some row does not see.
  auto step_on = [&](const uint8_t *buf, int base, auto kind) {
    constexpr bool EDGE = decltype(kind)::value;

    float s[TC][NT][4];
#pragma unroll
    for (int t = 0; t < TC; ++t) {
      const uint8_t *tile = buf + t * tile_bytes(D);
      uint32_t ka[D / 32], kb[D / 32], sa[2], sb[2];
      lds<D / 8>(tile + tile_k(D, g) + q4 * (D / 8), ka);
      lds<D / 8>(tile + tile_k(D, g + 8) + q4 * (D / 8), kb);
      if constexpr (D == 128) {
        const uint32_t x = e4m3x2(lds_u16(tile + tile_ks(D, g, 2 * q4)));
        const uint32_t y = e4m3x2(lds_u16(tile + tile_ks(D, g + 8, 2 * q4)));
        sa[0] = __byte_perm(x, x, 0x1010), sa[1] = __byte_perm(x, x, 0x3232);
        sb[0] = __byte_perm(y, y, 0x1010), sb[1] = __byte_perm(y, y, 0x3232);
      } else {
        const uint32_t x = lds_u8(tile + tile_ks(D, g, q4)), y = lds_u8(tile + tile_ks(D, g + 8, q4));
        sa[0] = e4m3x2(x * 0x101u), sb[0] = e4m3x2(y * 0x101u);
        sa[1] = sa[0], sb[1] = sb[0];
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t x[4], y[4];
        e2m1x8(ka[i], x);
        e2m1x8(kb[i], y);
        const uint32_t fa = sa[i >> 1], fb = sb[i >> 1];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = mul2(x[u], fa), y[u] = mul2(y[u], fb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t b[4];
          if constexpr (Sh::kQShared) {
            lds<16>(q_smem + ((nt * (KS / 2) + i) * 32 + lane) * 16, b);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) b[u] = qf[i][u];
          }
          if (i == 0)
            mma_f16_first(s[t][nt], x[0], y[0], x[1], y[1], b[0], b[1]);
          else
            mma_f16(s[t][nt], x[0], y[0], x[1], y[1], b[0], b[1]);
          mma_f16(s[t][nt], x[2], y[2], x[3], y[3], b[2], b[3]);
        }
      }
    }

    // masks and maxima
    bool rise = false;
    float top[NT][2];
    if constexpr (EDGE) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int hi = end_of(nt, k);
#pragma unroll
          for (int t = 0; t < TC; ++t)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int tok = base + 16 * t + 8 * b + g;
              const bool seen = tok < hi && (!a.window || tok >= hi - a.window);
              if (!seen) s[t][nt][2 * b + k] = -INFINITY;
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        top[nt][k] = fmaxf(s[0][nt][k], s[0][nt][2 + k]);
#pragma unroll
        for (int t = 1; t < TC; ++t) top[nt][k] = fmaxf(top[nt][k], fmaxf(s[t][nt][k], s[t][nt][2 + k]));
        rise |= top[nt][k] > bar_at[nt][k];
      }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 rs = scales[4 * nt];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = top[nt][k] * (k ? rs.y : rs.x);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float was = maximum(nt, k), up = fmaxf(was, x);
          const float f = was == -INFINITY ? 0.0f : fast_ex2(was - up);
          z[nt][k] = up == -INFINITY ? 0.0f : kLift - up;
          bar_at[nt][k] = (up + kLazy) / (k ? rs.y : rs.x);
          l[nt][k] *= f;
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[nt][i][k] *= f;
            o[nt][i][2 + k] *= f;
          }
        }
      }
    }

    // probabilities, as the second product's operand
    uint32_t pb[TC][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 rs = scales[4 * nt];
#pragma unroll
      for (int t = 0; t < TC; ++t) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float p0 = fast_ex2(fmaf(s[t][nt][2 * b], rs.x, z[nt][0]));
          const float p1 = fast_ex2(fmaf(s[t][nt][2 * b + 1], rs.y, z[nt][1]));
          l[nt][0] += p0;
          l[nt][1] += p1;
          pb[t][nt][b] = transpose8x8(pack2(p0, p1));
        }
      }
    }

#pragma unroll
    for (int t = 0; t < TC; ++t) {
      const uint8_t *tile = buf + t * tile_bytes(D);
      uint32_t v0[D / 32], v1[D / 32];           // tokens 2 q4, 2 q4 + 1 of the first and the second half
      lds<D / 8>(tile + tile_v(D, 2 * q4, g), v0);
      lds<D / 8>(tile + tile_v(D, 8 + 2 * q4, g), v1);
      const int group = g * (D / 8) / 16;
      uint32_t f0 = e4m3x2(lds_u16(tile + tile_vs(D, 2 * q4, group)));
      uint32_t f1 = e4m3x2(lds_u16(tile + tile_vs(D, 8 + 2 * q4, group)));
      if constexpr (EDGE) {
        // Tokens outside the tile's range hold nothing (a stale scale may be a NaN): they count 0.  A
        // scale that is a NaN inside it belongs to the rows that see its token alone, where 0 * NaN
        // would carry it to the others: it counts 0 too and then marks those rows' outputs.
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t &f = b ? f1 : f0;
            const int tok = base + 16 * t + 8 * b + 2 * q4 + e;
            const uint32_t part = e ? f >> 16 : f & 0xffffu;
            const bool in = tok >= lo_min && tok < hi_max, nan = (part & 0x7fffu) > 0x7c00u;
            if (!in || nan) f &= e ? 0x0000ffffu : 0xffff0000u;
            const uint32_t found = __ballot_sync(0xffffffffu, in && nan);
            if (found) {
              for (int x = 0; x < 4; ++x) {
                if (!((found >> (4 * g + x)) & 1)) continue;
                const int at = base + 16 * t + 8 * b + 2 * x + e;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int k = 0; k < 2; ++k)
                    if (const int hi = end_of(nt, k); at < hi && (!a.window || at >= hi - a.window))
#pragma unroll
                      for (int i = 0; i < KS; ++i) o[nt][i][k] = o[nt][i][2 + k] = __int_as_float(0x7fffffff);
              }
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t lo0[4], hi0[4], lo1[4], hi1[4];
        const uint32_t x0 = v0[i], y0 = v0[D / 64 + i], x1 = v1[i], y1 = v1[D / 64 + i];
        e2m1x8((x0 & 0x0f0f0f0fu) | ((y0 << 4) & 0xf0f0f0f0u), lo0);
        e2m1x8(((x0 >> 4) & 0x0f0f0f0fu) | (y0 & 0xf0f0f0f0u), hi0);
        e2m1x8((x1 & 0x0f0f0f0fu) | ((y1 << 4) & 0xf0f0f0f0u), lo1);
        e2m1x8(((x1 >> 4) & 0x0f0f0f0fu) | (y1 & 0xf0f0f0f0u), hi1);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t a0 = mul2(lo0[b], f0), a1 = mul2(hi0[b], f0), a2 = mul2(lo1[b], f1), a3 = mul2(hi1[b], f1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][4 * i + b], a0, a1, a2, a3, pb[t][nt][0], pb[t][nt][1]);
        }
      }
    }
  };

  int stage = 0;
  uint32_t phase = 0;
  bool alive = true;
  for (int c = w0; c < chunks; c += step) {
    if (!mbar_try(bar + 8 * stage, phase) && !mbar_wait(bar + 8 * stage, phase, abort)) {
      if (lane == 0) set_status(a.dev_status, DSPARK_ERR_DEVICE_TIMEOUT);
      alive = false;
      break;
    }
    const uint8_t *buf = smem + warp * Sh::kWarpBytes + stage * Sh::kStage;
    const int base = (c0 + c) * kChunk;
    if (base < lo_max || base + kChunk > hi_min)
      step_on(buf, base, std::true_type());
    else
      step_on(buf, base, std::false_type());
    __syncwarp();
    const int next = c + kStages * step;
    if (next < chunks) issue(next, stage, false);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!alive) {   // a wait gave up: the copies still on their way get one more bounded wait each
    for (int i = 0; i < kStages; ++i) {
      const long long t0 = clock64();
      while (!mbar_try(bar + 8 * stage, phase) && clock64() - t0 < kTimeoutCycles / 8) {
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }

  // what the loop had no registers for
  const volatile int *kept = reinterpret_cast<const volatile int *>(fixed);
  const int back[4] = {kept[8], kept[9], kept[10], kept[6]};
  // the CTA's warps meet
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x = l[nt][k];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      l[nt][k] = x;
      if (x != x && bar_at[nt][k] == -INFINITY) bar_at[nt][k] = 0.0f, z[nt][k] = kLift;   // every score was a NaN
      if (g == 0) {
        warp_m[warp * Sh::kRows + 8 * nt + 2 * q4 + k] = maximum(nt, k);
        warp_l[warp * Sh::kRows + 8 * nt + 2 * q4 + k] = x;
      }
    }
  __syncthreads();
  float *mine = reinterpret_cast<float *>(smem + warp * Sh::kWarpBytes);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int rr = 8 * nt + 2 * q4 + k;
      float big = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) big = fmaxf(big, warp_m[w * Sh::kRows + rr]);
      const float mine_m = maximum(nt, k), f = mine_m == -INFINITY ? 0.0f : fast_ex2(mine_m - big);
      // a thread's dimensions of a row: chunk g, in order
#pragma unroll
      for (int i = 0; i < KS; i += 2) {
        float4 v = make_float4(o[nt][i][k] * f, o[nt][i][2 + k] * f, o[nt][i + 1][k] * f, o[nt][i + 1][2 + k] * f);
        *reinterpret_cast<float4 *>(mine + rr * Sh::kOutRow + g * (D / 8) + 2 * i) = v;
      }
    }
  for (int rr = tid; rr < Sh::kRows; rr += kWarps * 32) {
    float big = -INFINITY, sum = 0.0f;
    for (int w = 0; w < kWarps; ++w) big = fmaxf(big, warp_m[w * Sh::kRows + rr]);
    for (int w = 0; w < kWarps; ++w)
      if (warp_m[w * Sh::kRows + rr] != -INFINITY)
        sum += warp_l[w * Sh::kRows + rr] * fast_ex2(warp_m[w * Sh::kRows + rr] - big);
    cta_m[rr] = big;
    cta_l[rr] = sum;
  }
  __syncthreads();
  constexpr int kVec = Sh::kRows * D / 4;            // float4 pieces of the tile's output
  float *acc = reinterpret_cast<float *>(smem);      // warp 0's partial becomes the CTA's
  for (int i = tid; i < kVec; i += kWarps * 32) {
    const int rr = i / (D / 4), d = 4 * (i % (D / 4));
    float4 v = *reinterpret_cast<float4 *>(acc + rr * Sh::kOutRow + d);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<float4 *>(smem + w * Sh::kWarpBytes + (rr * Sh::kOutRow + d) * 4);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    *reinterpret_cast<float4 *>(acc + rr * Sh::kOutRow + d) = v;
  }

  if (a.partial) {                                   // the parts meet in the merging kernel
    float *part = a.partial + (int64_t)blockIdx.x * Sh::kPartial;
    __syncthreads();
    if (tid < Sh::kRows) {
      part[tid] = cta_m[tid];
      part[Sh::kRows + tid] = cta_l[tid];
    }
    if (kept[7] > rank * kWarps)
      for (int i = tid; i < kVec; i += kWarps * 32)
        reinterpret_cast<float4 *>(part + 2 * Sh::kRows)[i] =
            *reinterpret_cast<const float4 *>(acc + i / (D / 4) * Sh::kOutRow + 4 * (i % (D / 4)));
    return;
  }

  // the cluster's CTAs meet: each takes its share of the output from all of them
  if (cs > 1)
    cluster.sync();
  else
    __syncthreads();
  for (int i = rank * kWarps * 32 + tid; i < kVec; i += cs * kWarps * 32) {
    const int rr = i / (D / 4), d = 4 * (i % (D / 4)), rho = back[2] + rr;
    if (rho >= back[1]) continue;
    float big = -INFINITY, sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int b = 0; b < cs; ++b) big = fmaxf(big, *cluster.map_shared_rank(cta_m + rr, b));
    for (int b = 0; b < cs; ++b) {
      const float mb = *cluster.map_shared_rank(cta_m + rr, b);
      if (mb == -INFINITY) continue;
      const float f = fast_ex2(mb - big);
      const float4 x = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(acc + rr * Sh::kOutRow + d, b));
      sum += *cluster.map_shared_rank(cta_l + rr, b) * f;
      v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y), v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
    }
    const float inv = big == -INFINITY ? 0.0f : a.out_scale / sum;
    const int64_t at = (int64_t)(back[0] + rho / a.group) * a.Hq + back[3] * a.group + rho % a.group;
    T y[4] = {Elem<DT>::from(v.x * inv), Elem<DT>::from(v.y * inv), Elem<DT>::from(v.z * inv),
              Elem<DT>::from(v.w * inv)};
    *reinterpret_cast<uint2 *>(reinterpret_cast<T *>(a.out) + at * D + d) = *reinterpret_cast<uint2 *>(y);
    if (a.lse && d == 0) a.lse[at] = big == -INFINITY ? -INFINITY : kLn2 * (big - kLift) + logf(sum);
  }
  if (cs > 1) cluster.sync();                        // no CTA leaves while another reads it
}

// Joins the parts of each row: a warp takes a row.
template <int DT, int D, int NT>
__global__ void __launch_bounds__(128) merge_kernel(const __grid_constant__ AttendArgs a, int row_tiles, int parts) {
  using T = typename Elem<DT>::T;
  constexpr int kRows = 8 * NT, kPartial = kRows * (D + 2), kLanes = D / 4;
  const int lane = threadIdx.x & 31, d = 4 * lane;
  const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int rr = (int)(job % kRows);
  int64_t unit = job / kRows;
  const float *part = a.partial + unit * parts * kPartial;
  const int rt = (int)(unit % row_tiles);
  unit /= row_tiles;
  const int h = (int)(unit % a.Hkv);
  grid_dep_launch();
  grid_dep_wait();
  if (unit / a.Hkv >= a.B || status_on_entry(a.dev_status)) return;
  const int64_t r = longest_first(a.kv_len, a.B, unit / a.Hkv, lane);
  const int64_t row0 = a.row_off[r], n = a.row_off[r + 1] - row0;
  const int64_t rho = (int64_t)rt * kRows + rr;
  if (rho >= n * a.group) return;
  float big = -INFINITY;
  for (int p = lane; p < parts; p += 32) big = fmaxf(big, part[p * kPartial + rr]);
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
  float sum = 0.0f;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p0 = 0; p0 < parts; p0 += 32) {
    // the lanes' factors of 32 parts, handed round
    float f = 0.0f, m = -INFINITY;
    if (p0 + lane < parts) {
      m = part[(p0 + lane) * kPartial + rr];
      f = m == -INFINITY ? 0.0f : fast_ex2(m - big);
      if (m != -INFINITY) sum = fmaf(part[(p0 + lane) * kPartial + kRows + rr], f, sum);
    }
    const uint32_t used = __ballot_sync(0xffffffffu, m != -INFINITY);
    for (int p = 0; p < min(32, parts - p0); ++p) {
      const float g = __shfl_sync(0xffffffffu, f, p);
      if (!((used >> p) & 1) || lane >= kLanes) continue;
      const float4 x = *reinterpret_cast<const float4 *>(part + (p0 + p) * kPartial + 2 * kRows + rr * D + d);
      v.x = fmaf(x.x, g, v.x), v.y = fmaf(x.y, g, v.y), v.z = fmaf(x.z, g, v.z), v.w = fmaf(x.w, g, v.w);
    }
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  const float inv = big == -INFINITY ? 0.0f : a.out_scale / sum;
  const int64_t at = (row0 + rho / a.group) * a.Hq + h * a.group + rho % a.group;
  if (lane < kLanes) {
    T y[4] = {Elem<DT>::from(v.x * inv), Elem<DT>::from(v.y * inv), Elem<DT>::from(v.z * inv),
              Elem<DT>::from(v.w * inv)};
    *reinterpret_cast<uint2 *>(reinterpret_cast<T *>(a.out) + at * D + d) = *reinterpret_cast<uint2 *>(y);
  }
  if (a.lse && lane == 0) a.lse[at] = big == -INFINITY ? -INFINITY : kLn2 * (big - kLift) + logf(sum);
}

// How a call is cut up.
struct Plan {
  int nt, row_tiles, parts;
  bool split;            // parts meet through the workspace and not in a cluster
  int64_t units;
};

Plan plan_of(int64_t B, int Hkv, int group, int D, int64_t len, int64_t max_rows, int64_t all_rows, int sms) {
  Plan p = {};
  const int64_t rows = max_rows * group, mean_rows = all_rows / B;
  // Tiles of 32 rows expand each stored element half as often as tiles of 16 but leave an SM 8 warps: better
  // where they are mostly full (one request with 32 row-heads 77 us against 87), worse where requests have
  // fewer rows than the largest (64 requests with 4 to 32: 90 us against 76).
  p.nt = rows <= 8 ? 1 : (rows <= 16 || D != 128 || mean_rows * group <= 24 ? 2 : 4);
  p.row_tiles = (int)((rows + 8 * p.nt - 1) / (8 * p.nt));
  p.units = B * Hkv * p.row_tiles;
  const int64_t slots = ctas_of(p.nt, D) * (int64_t)sms, least = kWarps * (int64_t)(4096 / D);   // tokens that give each warp a step
  p.parts = 1;
  while (p.parts < 8 && p.units * p.parts < slots && len >= 2 * p.parts * least) p.parts *= 2;
  // Few units with much to read: one wave of CTAs exactly, joined by a kernel of its own, where clusters of
  // eight leave most SMs idle (one row over 131071 tokens 44 us, 116 in clusters) or, with one or two
  // requests and so CTAs of one length, start a second wave (40 rows over 30000 tokens 83 us against 132).
  // Otherwise clusters are as fast or faster: 8 requests of up to 20000 tokens 35 us against 41.  A warp has
  // 8 steps at least, or the joining costs more than it gains (8000 tokens: 22 us against 12.6).
  const int64_t wave = slots / p.units, deep = len / (8 * least), n = wave < deep ? wave : deep;
  if (p.parts >= 4 && n > 1 && (n > p.parts || (B <= 2 && p.units * p.parts > slots))) p.parts = (int)(n < 1024 ? n : 1024), p.split = true;
  return p;
}

template <int DT, int D, int NT>
cudaError_t launch(const AttendArgs &a, const Plan &p, cudaStream_t s) {
  using Sh = Shape<D, NT>;
  auto *fn = attend_kernel<DT, D, NT>;
  cudaError_t e = ensure_dynamic_smem((const void *)fn, Sh::kSmem);
  if (e != cudaSuccess) return e;
  if (p.units * p.parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  e = launch_next(fn, p.units * p.parts, kWarps * 32, Sh::kSmem, p.split ? 1 : p.parts, s, a, p.row_tiles, p.parts);
  if (e != cudaSuccess || !p.split) return e;
  return launch_next(merge_kernel<DT, D, NT>, p.units * NT * 2, 128, 0, 1, s, a, p.row_tiles, p.parts);
}

template <int DT, int D>
cudaError_t launch_rows(const AttendArgs &a, const Plan &p, cudaStream_t s) {
  if constexpr (D == 128)
    if (p.nt == 4) return launch<DT, D, 4>(a, p, s);
  return p.nt == 1 ? launch<DT, D, 1>(a, p, s) : launch<DT, D, 2>(a, p, s);
}

}  // namespace

int64_t attend_workspace_bytes(int64_t B, int Hkv, int group, int D, int64_t len, int64_t max_rows, int64_t rows, int sms) {
  const Plan p = plan_of(B, Hkv, group, D, len, max_rows, rows, sms);
  return p.split ? p.units * p.parts * 8 * p.nt * (D + 2) * 4 : 0;
}

cudaError_t launch_attend(const AttendArgs &a, cudaStream_t s, int sms) {
  const Plan p = plan_of(a.B, a.Hkv, a.group, a.D, a.max_pages * a.page_size, a.max_rows, a.rows, sms);
  AttendArgs b = a;
  if (!p.split) b.partial = nullptr;
  if (a.dtype == DSPARK_BF16)
    return a.D == 128 ? launch_rows<DSPARK_BF16, 128>(b, p, s) : launch_rows<DSPARK_BF16, 64>(b, p, s);
  return a.D == 128 ? launch_rows<DSPARK_F16, 128>(b, p, s) : launch_rows<DSPARK_F16, 64>(b, p, s);
}

}  // namespace dspark
