// Attention of whole prompts: ragged rows of queries over ragged rows of keys and values in 16 bits.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - m),  lse = m + log sum_t p_t
// over the tokens t that a row sees: t < hi, hi = m_r (causal: m_r - n_r + j + 1 for row j of the n_r rows of a
// request with m_r tokens), and t >= hi - window with a window.  A row that sees nothing gets 0 and lse -inf.
//
// A CTA takes 256 row-heads (the query heads of one key/value head times the request's rows, two tiles of 128, so
// that grouped heads share each key and value that is loaded) and goes over the tokens 128 at a time:
//   warps 0-3, 4-7  one tile each: a thread has a row.  S comes out of tensor memory 32 columns at a time, and the
//                   probabilities go back over it in 16 bits, as the second product's left operand.
//   warp 8          allocates tensor memory (S and O of both tiles, 4 x 128 columns) and issues the products: S of
//                   a tile for the next tokens follows its P V, so that one tile's softmax runs beside the other's
//                   products.
//   warp 9          brings keys and values into a ring by tensor copies (128 tokens each).
//   warps 10, 11    look for infinities and NaN among the values of tokens that some rows do not see: a probability
//                   of 0 would carry them there.  They are taken out of the product and added at the end to
//                   the rows that see them.
//
// The running maximum moves only when a score passes it by 2^8, so that probabilities are computed against the
// maximum as it stands while they are checked; a warp with a row that passes takes its 32 rows again.
//
// Measured (one GB300): 16384 tokens, 32 query and 8 key/value heads of 128 dimensions, causal, 1682 us, 1308 TFLOP/s
// (1145 us at the rate of a large plain product); 16 prompts of 127 to 1021 tokens 140 us.  Bound by the chain of a tile
// (scores 512 cycles, softmax 1250, products 512, and the waits between them) of which two run beside each other, and
// for short prompts by what a CTA does before its first product (9000 cycles) and after its last (5000).  Two tiles
// that share loaded keys and values rather than one: each 32 KB that arrives serves 256 row-heads, and 512 columns of
// tensor memory hold just that.
//
// Rounding: scores, maxima, sums and outputs are fp32; probabilities are rounded to the type of the values (the
// product's two operands have one type), 2^-9 of each at most for bf16 and 2^-12 for fp16, which average out over
// tokens; the row's sum adds them unrounded.
#include <cuda.h>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace dspark {
namespace {

constexpr int kTokens = 128;               // of a step
constexpr int kTileRows = 128;
constexpr int kUnitRows = 2 * kTileRows;
constexpr int kThreads = 12 * 32;
constexpr float kLazy = 8.0f;              // how far (log2) a score may pass the running maximum

template <int D>
struct Shape {
  static constexpr int kPanels = D / 64;                       // of 64 dimensions: 128-byte rows
  static constexpr int kSlot = kTokens * D * 2;                // keys or values of a step
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kQ = kTileRows * D * 2;                 // of a tile
  static constexpr int kOffKv = 2 * kQ;
  static constexpr int kOffSh = kOffKv + kSlots * kSlot;
};

template <int SLOTS>
struct Shared {
  uint64_t full[SLOTS], empty[SLOTS], v_fine[SLOTS], q_full[2], s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int abort, skip, odd;                    // odd: values that are no numbers were taken out
  int64_t request, tile;
};

template <int D>
constexpr int smem_bytes() {
  return Shape<D>::kOffSh + (int)sizeof(Shared<Shape<D>::kSlots>) + 1024;
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory budget");

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tensor_g2s(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

template <int DT>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  uint32_t c;
  if constexpr (DT == DSPARK_BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(c) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(c) : "f"(hi), "f"(lo));
  return c;
}
// Whether one of a word's two elements is an infinity or a NaN, and the word with such elements 0.
template <int DT>
__device__ __forceinline__ bool odd_pair(uint32_t w) {
  constexpr uint32_t e = DT == DSPARK_BF16 ? 0x7f80u : 0x7c00u;
  return (w & e) == e || ((w >> 16) & e) == e;
}
template <int DT>
__device__ __forceinline__ uint32_t without_odd(uint32_t w) {
  constexpr uint32_t e = DT == DSPARK_BF16 ? 0x7f80u : 0x7c00u;
  if ((w & e) == e) w &= 0xffff0000u;
  if (((w >> 16) & e) == e) w &= 0x0000ffffu;
  return w;
}

__device__ __forceinline__ int end_of(const PromptArgs &a, int ctx, int kv, int rho) {
  return a.causal ? ctx + rho / a.group + 1 : kv;
}
__device__ __forceinline__ int start_of(const PromptArgs &a, int end) { return a.window ? max(end, a.window) - a.window : 0; }

// The token of a row-head among the first few (a CTA's): `on` / group, by a product, exact while on group is below 2^32.
__device__ __forceinline__ int token_of(const PromptArgs &a, int on) {
  return a.group > 1 ? (int)__umulhi((uint32_t)on, a.group_inv) : on;
}

// What a tile's row-heads see: from lo_max at the latest up to [hi_min, hi_max], in steps [t0, t1).
struct Tile {
  int lo_max, hi_min, hi_max, t0, t1;
  __device__ __forceinline__ bool on(int c) const { return c >= t0 && c < t1; }
  // whether a row does not see one of the step's tokens
  __device__ __forceinline__ bool edge(int c) const { return c * kTokens + kTokens > hi_min || c * kTokens < lo_max; }
  // the tokens of a step up to the last that is seen, in 32s
  __device__ __forceinline__ int columns(int c) const { return min(kTokens, (hi_max - c * kTokens + 31) / 32 * 32); }
  __device__ __forceinline__ void cut(int c0, int c1) {
    t0 = max(t0, c0);
    t1 = max(min(t1, c1), t0);
  }
};
__device__ __forceinline__ Tile tile_of(const PromptArgs &a, int ctx, int kv, int first, int total) {
  Tile t;
  t.hi_min = end_of(a, ctx, kv, first);
  t.hi_max = end_of(a, ctx, kv, min(first + kTileRows, total) - 1);
  t.lo_max = start_of(a, t.hi_max);
  t.t0 = start_of(a, t.hi_min) / kTokens;
  t.t1 = max(t.hi_max <= 0 ? 0 : (t.hi_max + kTokens - 1) / kTokens, t.t0);
  return t;
}

// A request's units lie from row_off[r] group / 256 + r on: as many places as it may need, with no sum over the
// requests before it.  The last r whose units begin at or before `unit`, by one warp.
__device__ __forceinline__ int64_t request_of_unit(const int32_t *row_off, int64_t B, int group, int64_t unit, int lane) {
  int64_t lo = 0, len = B;
  while (len > 1) {
    const int64_t step = (len + 31) >> 5, at = lane * step;
    const bool in = at < len && (int64_t)row_off[lo + at] * group / kUnitRows + lo + at <= unit;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const int64_t last = m ? 31 - __clz(m) : 0, end = lo + len;
    lo += last * step;
    len = end - lo < step ? end - lo : step;
  }
  return lo;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A step's scores as probabilities 2^(s R + z) in 16 bits, their sum and the largest exponent.  The next 32 scores are on
// their way while 32 are worked on.  EDGE: only columns lo .. hi - 1 are seen, and those from `cols` on not looked at.
template <int DT, bool EDGE>
__device__ __forceinline__ void take_step(uint32_t s_at, int cols, int lo, int hi, float R, float z, uint32_t (&P)[64],
                                          float &most, float &sum) {
  const unsigned long long R2 = f2_pack(R, R), z2 = f2_pack(z, z);
  unsigned long long total[2] = {0, 0};
  float top[2] = {-INFINITY, -INFINITY};
  uint32_t s[2][32];
  tmem_ld32(s_at, s[0]);
  tmem_wait_ld(s[0]);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (EDGE && b * 32 >= cols) break;
    if (b < 3 && (!EDGE || b * 32 + 32 < cols)) tmem_ld32(s_at + b * 32 + 32, s[(b + 1) & 1]);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const int i = k / 2 & 1;
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[b & 1][k]), __uint_as_float(s[b & 1][k + 1])), R2, z2), x0, x1);
      if (EDGE) {
        const int tok = b * 32 + k;
        if (!(tok < hi && tok >= lo)) x0 = -INFINITY;
        if (!(tok + 1 < hi && tok + 1 >= lo)) x1 = -INFINITY;
      }
      top[i] = max3(top[i], x0, x1);
      const float p0 = fast_ex2(x0), p1 = fast_ex2(x1);
      total[i] = f2_add(total[i], f2_pack(p0, p1));
      P[b * 16 + k / 2] = pack_pair<DT>(p0, p1);
    }
    if (EDGE) __syncwarp();
    if (b < 3 && (!EDGE || b * 32 + 32 < cols)) tmem_wait_ld(s[(b + 1) & 1]);
  }
  most = fmaxf(top[0], top[1]);
  float t0, t1;
  f2_unpack(f2_add(total[0], total[1]), t0, t1);
  sum = t0 + t1;
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  using T = typename Elem<DT>::T;
  using Sh = Shape<D>;
  constexpr int kSlots = Sh::kSlots;
  constexpr float kLift = DT == DSPARK_F16 ? 6.0f : 0.0f;   // fp16 probabilities are kept 2^6 up: small ones stay normal
  // fp32 sums; bf16 or fp16 operands, queries and keys K-major, values MN-major; M = 128
  constexpr uint32_t kType = DT == DSPARK_BF16 ? (1u << 7) | (1u << 10) : 0u;
  constexpr uint32_t kIdesc = (1u << 4) | kType | ((uint32_t)(kTileRows >> 4) << 24);
  constexpr uint32_t kIdescO = kIdesc | (1u << 16) | ((uint32_t)(D >> 3) << 17);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sb = (raw + 1023u) & ~1023u;
  uint8_t *gb = smem_raw + (sb - raw);
  Shared<kSlots> &sh = *reinterpret_cast<Shared<kSlots> *>(gb + Sh::kOffSh);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort = &sh.abort;

  // the CTA's unit, last ones (of a causal prompt: the longest) first
  const int h = (int)(blockIdx.x % (unsigned)a.Hkv);
  const int64_t at = blockIdx.x / (unsigned)a.Hkv;
  const int part = (int)(at % a.parts);
  const int64_t unit = a.units - 1 - at / a.parts;
  if (warp == 0) {
    const int64_t r = request_of_unit(a.row_off, a.B, a.group, unit, lane);
    if (lane == 0) {
      sh.request = r;
      sh.tile = unit - ((int64_t)a.row_off[r] * a.group / kUnitRows + r);
    }
  } else if (warp == 1) {                                        // beside the search
    if (lane < kSlots) {
      mbar_init(smem_u32(&sh.full[lane]), 1);
      mbar_init(smem_u32(&sh.empty[lane]), 3);                   // the products and both looking warps
      mbar_init(smem_u32(&sh.v_fine[lane]), 2);
    }
    if (lane < 2) {
      mbar_init(smem_u32(&sh.q_full[lane]), kTileRows);
      mbar_init(smem_u32(&sh.s_full[lane]), 1);
      mbar_init(smem_u32(&sh.p_full[lane]), 4);
      mbar_init(smem_u32(&sh.o_full[lane]), 1);
    }
    if (lane == 0) {
      mbar_init(smem_u32(&sh.drain), 1);
      sh.abort = sh.odd = 0;
      sh.skip = read_status(a.dev_status);
    }
    __syncwarp();
    fence_barrier_init();
  }
  __syncthreads();
  if (sh.skip) return;
  const int64_t r = sh.request;
  const int64_t row0 = a.row_off[r], row1 = a.row_off[r + 1], kv0 = a.kv_off[r], kv1 = a.kv_off[r + 1];
  if (row0 < 0 || row1 < row0 || row1 > a.rows || kv0 < 0 || kv1 < kv0 || kv1 > a.kv_rows) {
    if (threadIdx.x == 0) set_status(a.dev_status, DSPARK_ERR_OFFSETS);
    return;
  }
  const int n = (int)(row1 - row0), kv = (int)(kv1 - kv0), ctx = kv - n, total = n * a.group;
  if (sh.tile < 0 || sh.tile * kUnitRows >= total) return;      // a place that its request has no need of
  const int first = (int)sh.tile * kUnitRows, tiles = total - first > kTileRows ? 2 : 1;

  // the tiles and their steps, and the CTA's steps
  Tile tile_a = tile_of(a, ctx, kv, first, total), tile_b = tile_a;
  tile_b.t1 = tile_b.t0;
  int c0 = tile_a.t0, c1 = tile_a.t1;
  if (tiles == 2) {
    tile_b = tile_of(a, ctx, kv, first + kTileRows, total);
    c0 = min(c0, tile_b.t0);
    c1 = max(c1, tile_b.t1);
  }
  if (a.parts > 1) {                                             // this part's share of them
    const int all = max(c1 - c0, 0), from = c0 + (int)((int64_t)all * part / a.parts);
    c1 = c0 + (int)((int64_t)all * (part + 1) / a.parts);
    c0 = from;
    tile_a.cut(c0, c1);
    tile_b.cut(c0, c1);
  }
  // an edge of either tile (a row past the last sees nothing, and keeps nothing)
  auto any_edge = [&](int c) { return (tile_a.on(c) && tile_a.edge(c)) || (tile_b.on(c) && tile_b.edge(c)); };

  if (warp == 8) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;                                 // S0, S1, O0, O1: 128 columns each
  const uint32_t full = smem_u32(sh.full), empty = smem_u32(sh.empty);

  if (warp == 9) {
    // ---------------- keys and values ----------------
    // In the order in which they are used: K of the first step, then K of the next and V of each.
    if (lane == 0 && c0 < c1) {
      int idx = 0;
      auto bring = [&](const CUtensorMap *map, int x, int z, int c) {
        const int s = idx % kSlots;
        if (!mbar_wait(empty + 8 * s, (uint32_t)(idx / kSlots & 1) ^ 1u, abort)) return false;
        mbar_arrive_tx(full + 8 * s, Sh::kSlot);
#pragma unroll
        for (int p = 0; p < Sh::kPanels; ++p)
          tensor_g2s(sb + Sh::kOffKv + s * Sh::kSlot + p * (kTokens * 128), map, x + p * 64, (int)kv0 + c * kTokens, z, full + 8 * s);
        ++idx;
        return true;
      };
      const int kx = h * a.k_x, kz = h * a.k_z, vx = h * a.v_x, vz = h * a.v_z;
      bool ok = bring(&k_map, kx, kz, c0);
      for (int c = c0; ok && c < c1; ++c) {
        if (c + 1 < c1) ok = bring(&k_map, kx, kz, c + 1);
        if (ok) ok = bring(&v_map, vx, vz, c);
      }
      if (!ok)                                                   // no copy may be under way at the end
        for (int i = max(idx - kSlots, 0); i < idx; ++i) {
          const long long begun = clock64();
          while (!mbar_try(full + 8 * (i % kSlots), (uint32_t)(i / kSlots & 1)) && clock64() - begun < kTimeoutCycles / 8) {
          }
        }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---------------- products ----------------
    // (the whole warp waits, one lane issues)
    if (c0 < c1) {
      bool ok = true;
      int fine = 0;                                              // edges whose values have been looked at
      auto wait = [&](uint64_t &bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try(smem_u32(&bar), parity) || mbar_wait(smem_u32(&bar), parity, abort)) != 0;
      };
      auto slot_full = [&](int idx) { return wait(sh.full[idx % kSlots], (uint32_t)(idx / kSlots & 1)); };
      const uint64_t q_desc = smem_desc(sb, 16, 1024), k_desc = smem_desc(sb + Sh::kOffKv, 16, 1024),
                     v_desc = smem_desc(sb + Sh::kOffKv, kTokens * 128, 1024);
      auto scores = [&](const Tile &tile, int i, int c, int idx) {   // S of tile i for step c, keys in slot idx
        const uint64_t k_at = desc_on(k_desc, (idx % kSlots) * Sh::kSlot), q_at = desc_on(q_desc, i * Sh::kQ);
        const uint32_t idesc = kIdesc | ((uint32_t)(tile.columns(c) >> 3) << 17);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t on = s / 4 * (kTileRows * 128) + s % 4 * 32;     // (tiles and steps have 128 rows both)
            mma_bf16(tmem + i * 128, desc_on(q_at, on), desc_on(k_at, on), idesc, s > 0);
          }
          mma_commit(smem_u32(&sh.s_full[i]));
        }
        __syncwarp();
      };
      auto give_back = [&](int idx) {
        if (elect_one()) mma_commit(empty + 8 * (idx % kSlots));
        __syncwarp();
      };
      for (int i = 0; ok && i < tiles; ++i) ok = wait(sh.q_full[i], 0);
      if (ok) ok = slot_full(0);
      tc_fence_after();
      if (ok) {
        if (tile_a.on(c0)) scores(tile_a, 0, c0, 0);
        if (tile_b.on(c0)) scores(tile_b, 1, c0, 0);
        give_back(0);
      }
      uint32_t turn[2] = {0, 0};
      for (int c = c0; ok && c < c1; ++c) {
        const int j = c - c0, k_idx = 1 + 2 * j, v_idx = c + 1 < c1 ? 2 + 2 * j : 1 + 2 * j;
        const uint64_t v_at = desc_on(v_desc, (v_idx % kSlots) * Sh::kSlot);
        bool v_there = false, k_there = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Tile &tile = i ? tile_b : tile_a;
          if (ok && tile.on(c)) {
            if (!v_there) {
              ok = slot_full(v_idx);
              if (ok && any_edge(c)) {
                ok = wait(sh.v_fine[fine % kSlots], (uint32_t)(fine / kSlots & 1));
                ++fine;
              }
              v_there = true;
            }
            if (ok) ok = wait(sh.p_full[i], turn[i]);
            turn[i] ^= 1;
            if (ok) {
              tc_fence_after();
              const int steps = tile.columns(c) / 16;
              if (elect_one()) {
#pragma unroll
                for (int s = 0; s < kTokens / 16; ++s)
                  if (s < steps)
                    mma_ts(tmem + 256 + i * 128, tmem + i * 128 + s * 8, desc_on(v_at, s * 2048), kIdescO, c > tile.t0 || s > 0);
                if (c + 1 == tile.t1) mma_commit(smem_u32(&sh.o_full[i]));
              }
              __syncwarp();
            }
          }
          if (ok && c + 1 < c1 && tile.on(c + 1)) {
            if (!k_there) ok = slot_full(k_idx);
            k_there = true;
            tc_fence_after();
            if (ok) scores(tile, i, c + 1, k_idx);
          }
        }
        if (ok) {
          if (!v_there) ok = slot_full(v_idx);                   // (a step that no tile takes)
          if (ok && c + 1 < c1 && !k_there) ok = slot_full(k_idx);
          if (c + 1 < c1) give_back(k_idx);
          give_back(v_idx);
        }
      }
      if (!ok && lane == 0) {
        set_status(a.dev_status, DSPARK_ERR_DEVICE_TIMEOUT);
        mma_commit(smem_u32(&sh.drain));
        const long long begun = clock64();
        while (!mbar_try(smem_u32(&sh.drain), 0) && clock64() - begun < kTimeoutCycles / 8) {
        }
      }
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------- values that are no numbers ----------------
    // These warps go through every slot of the ring, edges or not, and give it back too: a wait for a phase that
    // does not follow on the last one seen could take an older one for it.
    int fine = 0;
    const int uses = c1 > c0 ? 2 * (c1 - c0) : 0;
    for (int idx = 0; idx < uses; ++idx) {
      const int slot = idx % kSlots;
      const bool ok = mbar_wait(full + 8 * slot, (uint32_t)(idx / kSlots & 1), abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      // slots hold K0, K1, V0, K2, V1, ...: the step whose values this is
      const int c = idx == uses - 1 ? c1 - 1 : ((idx & 1) || idx == 0 ? -1 : c0 + idx / 2 - 1);
      if (c >= 0 && any_edge(c)) {
        uint4 *v = reinterpret_cast<uint4 *>(gb + Sh::kOffKv + slot * Sh::kSlot);
        bool found = false;
#pragma unroll 8
        for (int i = threadIdx.x - 320; i < Sh::kSlot / 16; i += 64) {
          const uint4 x = v[i];
          if (odd_pair<DT>(x.x) || odd_pair<DT>(x.y) || odd_pair<DT>(x.z) || odd_pair<DT>(x.w)) {
            v[i] = make_uint4(without_odd<DT>(x.x), without_odd<DT>(x.y), without_odd<DT>(x.z), without_odd<DT>(x.w));
            found = true;
          }
        }
        if (found) sh.odd = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.v_fine[fine % kSlots]));
        ++fine;
      }
      if (lane == 0) mbar_arrive(empty + 8 * slot);
      __syncwarp();
    }
  } else {
    // ---------------- softmax: a thread has a row of its warpgroup's tile ----------------
    const int i = warp >> 2, t = threadIdx.x & 127, q4 = warp & 3;
    const Tile tile = i ? tile_b : tile_a;
    if (i < tiles) {
      // queries: 16 bytes at a time, neighbouring threads along a row, all of a thread's loads under way
      const T *q = reinterpret_cast<const T *>(a.q) + (int64_t)h * a.group * a.q_head;
      constexpr int kPieces = D / 8;
      const int skipped = first / a.group * a.group;             // row-heads of tokens before the CTA's first
      const int64_t q_row0 = row0 + first / a.group;
      {
        uint4 x[kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          const int p = t + u * kTileRows, rho = first + i * kTileRows + p / kPieces;
          const int on = rho - skipped, tok = token_of(a, on);
          x[u] = make_uint4(0, 0, 0, 0);
          if (rho < total)
            x[u] = __ldg(reinterpret_cast<const uint4 *>(q + (q_row0 + tok) * a.q_row + (int64_t)(on - tok * a.group) * a.q_head +
                                                         p % kPieces * 8));
        }
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          const int p = t + u * kTileRows, row = p / kPieces, c = p % kPieces;
          *reinterpret_cast<uint4 *>(gb + i * Sh::kQ + c / 8 * (kTileRows * 128) + row * 128 + ((c % 8) ^ (row & 7)) * 16) = x[u];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&sh.q_full[i]));

      const int rho = first + i * kTileRows + t;
      const bool real = rho < total;
      const int end = real ? end_of(a, ctx, kv, rho) : 0, start = start_of(a, end);
      const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
      const uint32_t s_at = tmem + lanes + i * 128, o_at = tmem + lanes + 256 + i * 128;
      const float R = a.scale_log2;
      // Probabilities are 2^(s R + z), z = kLift - the running maximum; none yet: -inf and z = 0.  The first step measures
      // its maximum: against a reference of 0, which near enough scores would allow and which saves 1300 cycles, the
      // largest probability is no power of two and rounded too (bf16 outputs 2.2e-3 off and not 1.8e-3 to 2.0e-3).
      float top = -INFINITY, z = 0.0f, l = 0.0f;
      uint32_t turn = 0;
      bool ok = true;
      for (int c = tile.t0; c < tile.t1; ++c) {
        ok = mbar_try(smem_u32(&sh.s_full[i]), turn) || mbar_wait(smem_u32(&sh.s_full[i]), turn, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        turn ^= 1;
        tc_fence_after();
        const bool at_edge = tile.edge(c);
        const int cols = tile.columns(c), lo = start - c * kTokens, hi = end - c * kTokens;
        bool measure = c == tile.t0;
        uint32_t P[64];
        float more;
        for (;;) {
          if (measure) {
            float most = -INFINITY;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              if (b * 32 >= cols) break;
              uint32_t s[32];
              tmem_ld32(s_at + b * 32, s);
              tmem_wait_ld(s);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const int tok = b * 32 + k;
                const float x = __uint_as_float(s[k]) * R;
                if (!at_edge || (tok < hi && tok >= lo)) most = fmaxf(most, x);
              }
              __syncwarp();
            }
            const float up = fmaxf(top, most);
            const float f = top == -INFINITY ? 0.0f : fast_ex2(top - up);
            const bool risen = up > top;
            if (c > tile.t0 && __any_sync(0xffffffffu, risen)) {
              // O of the steps before is complete: S of this one came after it
#pragma unroll 1
              for (int b = 0; b < D / 32; ++b) {
                uint32_t o[32];
                tmem_ld32(o_at + b * 32, o);
                tmem_wait_ld(o);
                if (risen)
#pragma unroll
                  for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                __syncwarp();
                tmem_st32(o_at + b * 32, o);
              }
              tmem_wait_st();
            }
            if (risen) {
              l *= f;
              top = up;
              z = kLift - up;
            }
            __syncwarp();
          }
          float most;
          if (at_edge)
            take_step<DT, true>(s_at, cols, lo, hi, R, z, P, most, more);
          else
            take_step<DT, false>(s_at, kTokens, 0, 0, R, z, P, most, more);
          // (a first maximum of -inf leaves the next step to measure; an infinite score measured leaves it at that)
          if (measure || !__any_sync(0xffffffffu, most > kLift + kLazy || (top == -INFINITY && most > -INFINITY))) break;
          measure = true;
        }
        l += more;
        // P over S
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b * 64 >= cols) break;
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) w[k] = P[b * 32 + k];
          tmem_st32(s_at + b * 32, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[i]));
        __syncwarp();
      }
      // ---------------- the row's output ----------------
      const bool none = tile.t1 <= tile.t0;
      if (ok && !none) {
        ok = mbar_wait(smem_u32(&sh.o_full[i]), 0, abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
      if (ok) {
        const int tok = real ? rho / a.group : 0;
        const int64_t to = (row0 + tok) * a.Hq + h * a.group + (rho - tok * a.group);
        const bool odd = *(volatile int *)&sh.odd != 0, split = a.parts > 1;
        const float inv = split ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
        float *partial = split ? a.partial + ((int64_t)part * a.rows * a.Hq + to) * (D + 2) : nullptr;
#pragma unroll 1                                                 // (unrolled, the code comes into the cache late)
        for (int b = 0; b < D / 32; ++b) {
          __syncwarp();                                          // (the load takes the warp together)
          uint32_t o[32];
          if (none) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          } else {
            tmem_ld32(o_at + b * 32, o);
            tmem_wait_ld(o);
          }
          if (real) {
            float y[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = l == 0.0f ? 0.0f : __uint_as_float(o[k]) * inv;
            if (odd)                                             // values that were taken out of the product
              for (int c = tile.t0; c < tile.t1; ++c) {
                if (!any_edge(c)) continue;
                for (int x = max(start, c * kTokens); x < min(end, c * kTokens + kTokens); ++x) {
                  const T *v = reinterpret_cast<const T *>(a.v) + (kv0 + x) * a.v_row + h * a.v_head + b * 32;
#pragma unroll
                  for (int k = 0; k < 32; ++k) {
                    const float u = Elem<DT>::to(v[k]);
                    if (!(fabsf(u) <= 3.4e38f)) y[k] += u;
                  }
                }
              }
            if (split) {
#pragma unroll
              for (int k = 0; k < 32; k += 2) *reinterpret_cast<float2 *>(partial + 2 + b * 32 + k) = make_float2(y[k], y[k + 1]);
            } else {                                             // into the place of the tile's queries, swizzled by the row
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4 *>(gb + i * Sh::kQ + t * (2 * D) + ((b * 4 + k) ^ (t & 7)) * 16) =
                    make_uint4(pack_pair<DT>(y[8 * k], y[8 * k + 1]), pack_pair<DT>(y[8 * k + 2], y[8 * k + 3]),
                               pack_pair<DT>(y[8 * k + 4], y[8 * k + 5]), pack_pair<DT>(y[8 * k + 6], y[8 * k + 7]));
            }
          }
        }
        __syncwarp();
        if (!split) {                                            // whole rows at a time: the warp's 32
          constexpr int kLanes = D / 8;
          const int skipped = first / a.group * a.group;
          T *out = reinterpret_cast<T *>(a.out) + ((row0 + first / a.group) * a.Hq + h * a.group) * D;
#pragma unroll
          for (int x = lane; x < 32 * kLanes; x += 32) {
            const int row = q4 * 32 + x / kLanes, piece = x % kLanes, rho2 = first + i * kTileRows + row;
            const int on = rho2 - skipped, tok2 = token_of(a, on);
            if (rho2 < total)
              *reinterpret_cast<uint4 *>(out + ((int64_t)tok2 * a.Hq + on - tok2 * a.group) * D + piece * 8) =
                  *reinterpret_cast<const uint4 *>(gb + i * Sh::kQ + row * (2 * D) + (piece ^ (row & 7)) * 16);
          }
        }
        if (real) {
          if (split)
            *reinterpret_cast<float2 *>(partial) = make_float2(top, l);
          else if (a.lse)
            a.lse[to] = l == 0.0f ? -INFINITY : kLn2 * (top == -INFINITY ? 0.0f : top - kLift) + logf(l);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// Joins the parts of each row: a warp takes a row-head.
template <int DT, int D>
__global__ void __launch_bounds__(128) prompt_join(const __grid_constant__ PromptArgs a) {
  using T = typename Elem<DT>::T;
  constexpr int kLift = DT == DSPARK_F16 ? 6 : 0, kMine = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= a.rows * a.Hq || read_status(a.dev_status) || row / a.Hq < a.row_off[0] || row / a.Hq >= a.row_off[a.B]) return;
  const float *part = a.partial + row * (D + 2);
  const int64_t step = a.rows * a.Hq * (D + 2);
  float m = -INFINITY, own_l = 0.0f;                              // lane p has part p: at most 32
  if (lane < a.parts) {
    const float2 ml = *reinterpret_cast<const float2 *>(part + lane * step);
    m = ml.x, own_l = ml.y;
  }
  float big = m;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
  // (a part whose every score was a NaN has no maximum but a sum)
  const float f = own_l == 0.0f ? 0.0f : (m == -INFINITY || big == -INFINITY ? 1.0f : fast_ex2(m - big));
  float sum = own_l * f;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  float y[kMine] = {};
  for (int p = 0; p < a.parts; ++p) {
    const float g = __shfl_sync(0xffffffffu, f, p);
    if (g == 0.0f) continue;
    const float2 *o = reinterpret_cast<const float2 *>(part + p * step + 2 + lane * kMine);
#pragma unroll
    for (int k = 0; k < kMine; k += 2) {
      const float2 u = o[k / 2];
      y[k] = fmaf(u.x, g, y[k]);
      y[k + 1] = fmaf(u.y, g, y[k + 1]);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  T *to = reinterpret_cast<T *>(a.out) + row * D + lane * kMine;
#pragma unroll
  for (int k = 0; k < kMine; k += 2) *reinterpret_cast<uint32_t *>(to + k) = pack_pair<DT>(y[k] * inv, y[k + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = sum == 0.0f ? -INFINITY : kLn2 * (big == -INFINITY ? 0.0f : big - kLift) + logf(sum);
}

// Keys or values as a tensor that copies of 128 rows by 64 dimensions are taken from: heads inside the rows as one
// long row (a head is a place along it), rows inside the heads as [head][row][dim].  The copies' strides have to be
// multiples of one another, which either form is by itself.
bool heads_in_rows(int64_t rows, int Hkv, int D, int64_t row, int64_t head) {
  return rows < 2 || Hkv < 2 || (Hkv - 1) * head + D <= row;
}
bool encode(CUtensorMap *map, const void *data, const PromptArgs &a, int64_t row, int64_t head, int *x_step, int *z_step) {
  static decltype(&cuTensorMapEncodeTiled) fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (decltype(&cuTensorMapEncodeTiled))p;
  }();
  if (!fn) return false;
  const bool in_rows = heads_in_rows(a.kv_rows, a.Hkv, a.D, row, head);
  const int64_t wide = in_rows ? (a.Hkv - 1) * head + a.D : a.D;
  if (a.kv_rows < 2) row = wide;
  const cuuint64_t dims[3] = {(cuuint64_t)wide, (cuuint64_t)a.kv_rows, (cuuint64_t)(in_rows ? 1 : a.Hkv)};
  const cuuint64_t strides[2] = {(cuuint64_t)row * 2, (cuuint64_t)(in_rows ? row : head) * 2};
  const cuuint32_t box[3] = {64, kTokens, 1}, unit[3] = {1, 1, 1};
  *x_step = in_rows ? (int)head : 0;
  *z_step = in_rows ? 0 : 1;
  return fn(map, a.dtype == DSPARK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, (void *)data, dims,
            strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Parts of each unit's tokens, where the units are too few to fill the SMs: at least 4 steps a part.
int parts_of(int64_t units, int64_t kv_rows, int64_t B, int sms) {
  const int64_t room = units > 0 ? sms / units : 1, deep = (kv_rows + B * kTokens - 1) / (B * kTokens) / 4;
  const int64_t p = room < deep ? room : deep;
  return (int)(p < 2 ? 1 : (p < 32 ? p : 32));
}

template <int DT, int D>
cudaError_t launch(const PromptArgs &a, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s) {
  auto *fn = prompt_kernel<DT, D>;
  const cudaError_t e = ensure_dynamic_smem((const void *)fn, smem_bytes<D>());
  if (e != cudaSuccess) return e;
  const int64_t grid = a.units * a.parts * a.Hkv;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  fn<<<(unsigned)grid, kThreads, smem_bytes<D>(), s>>>(a, k, v);
  if (a.parts > 1) prompt_join<DT, D><<<(unsigned)((a.rows * a.Hq + 3) / 4), 128, 0, s>>>(a);
  return cudaGetLastError();
}

int64_t units_of(int64_t rows, int64_t B, int group) { return rows * group / kUnitRows + B; }

}  // namespace

int64_t prompt_workspace_bytes(int64_t rows, int64_t kv_rows, int64_t B, int Hq, int Hkv, int D, int sms) {
  const int p = parts_of(units_of(rows, B, Hq / Hkv) * Hkv, kv_rows, B, sms);
  return p > 1 ? p * rows * Hq * (D + 2) * 4 : 0;
}

bool prompt_layout_ok(int64_t kv_rows, int Hkv, int D, int64_t row, int64_t head) {
  constexpr int64_t most = (int64_t)1 << 38;
  if (kv_rows > 1 && (row < 1 || row >= most)) return false;
  if (Hkv > 1 && (head < 1 || head >= most)) return false;
  return heads_in_rows(kv_rows, Hkv, D, row, head) ? (Hkv - 1) * head + D <= 0x7fffffff : head % row == 0;
}

cudaError_t launch_prompt(const PromptArgs &args, cudaStream_t s, int sms) {
  PromptArgs a = args;
  a.units = units_of(a.rows, a.B, a.group);
  a.parts = parts_of(a.units * a.Hkv, a.kv_rows, a.B, sms);
  a.group_inv = a.group > 1 ? 0xffffffffu / (unsigned)a.group + 1 : 0;
  CUtensorMap k = {}, v = {};
  if (a.kv_rows > 0 && (!encode(&k, a.k, a, a.k_row, a.k_head, &a.k_x, &a.k_z) ||
                        !encode(&v, a.v, a, a.v_row, a.v_head, &a.v_x, &a.v_z)))
    return cudaErrorInvalidValue;
  if (a.dtype == DSPARK_BF16) return a.D == 128 ? launch<DSPARK_BF16, 128>(a, k, v, s) : launch<DSPARK_BF16, 64>(a, k, v, s);
  return a.D == 128 ? launch<DSPARK_F16, 128>(a, k, v, s) : launch<DSPARK_F16, 64>(a, k, v, s);
}

}  // namespace dspark
