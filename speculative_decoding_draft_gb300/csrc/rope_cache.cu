// Norm and position rotation of query and key heads, the append of rotated keys and of values to
// the paged cache in 4 bits, and the cache's read-back.
//
//   y = x rsqrt(mean(x^2) + eps) w          (one head of D dimensions, where a weight is given)
//   (a, b) -> g (a c - b s, b c + a s),     c, s = cos, sin of position * inv_freq_i
//   scale = e4m3(max |y| / 6), element = e2m1(y / scale)       (16 dimensions; append only)
//
// Angles.  A frequency is kept as the fraction of a turn per position in 64-bit fixed point; the
// product with the position wraps modulo 2^64, which is modulo a whole turn, so the angle of a
// position in the millions is as exact as that of position 1 (an fp32 product would be off by 0.06
// radians at position 2^20).
//
// All arithmetic is in fp32; the queries (and the keys of norm_rope) are rounded once, the keys
// and values that go to the cache once to 4 bits.
//
// A warp takes one row, or one of `parts` equal shares of its heads, by itself: it brings the heads
// into a ring of its own with bulk copies, all of a usual row under way at once, finds the row's place
// and angles meanwhile, keeps cosines and sines in registers and goes over the heads.  A lane holds 8
// neighbouring dimensions of a head, a head takes D/8 lanes, and the partner of the half layout lies
// rot/16 lanes away; with every dimension's cosine and signed sine both layouts are x C + partner S.
// Arithmetic goes in pairs of fp32 (one instruction for two).
//
// Bound by the latency of its loads until these are all in flight: with two 16-byte loads a lane ahead
// in registers the append of 9216 rows with 48 heads of 128 dimensions took 75 us, at 30 % of the
// memory's rate and 44 % of the issue slots.  Now 63 us, with 71 % of the issue slots.
#include "heads.cuh"

namespace dspark {
namespace {

// Ring of a warp and CTAs an SM: the append, with more to compute, wants warps rather than bytes under way.
constexpr int ring_bytes(bool append) { return append ? 4096 : 6144; }
constexpr int kEnoughWarps = 2048; // 13 on each of 152 SMs, under half of those that fit there together
constexpr int kWarps = 4;          // of a CTA; they share nothing

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN stays
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float c;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// One lane's 8 elements of a group of 16 as codes, and the group's scale.  The lane beside holds the others;
// unit is a power of two, inv = 1 / unit.
//
// Both quotients, by 6 and by the scale, are correctly rounded: the product with the reciprocal and one step of
// the remainder, which fp32 holds exactly as the divisor has 4 bits at most.  A quotient that is no border of
// two codes (or scales) lies at least half a step of fp32 off it and does not round to it, so what is stored
// is the nearest to y, for normed and turned keys with all the bits of fp32 as for 16-bit values.
__device__ __forceinline__ uint32_t quantize8(const Pair (&x)[4], float inv, float unit, uint8_t *scale) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = floats_of(x[i]);
    top = max_nan(top, max_nan(fabsf(f.x), fabsf(f.y)));
  }
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  // a NaN stays one; what the largest scale is too small for (infinities among it) is cut to where the
  // remainder is finite
  const float most = min_nan(top * inv, 1048576.0f);
  const float about = most * (1.0f / 6.0f);
  const float sixth = fmaf(fmaf(about, -6.0f, most), 1.0f / 6.0f, about);
  const __nv_fp8_storage_t s8 = __nv_cvt_float_to_fp8(sixth, __NV_SATFINITE, __NV_E4M3);
  *scale = s8;
  // 0 (nothing to keep) and NaN (nothing else to say) leave the elements 0
  if ((s8 & 0x7f) == 0 || (s8 & 0x7f) == 0x7f) return 0;
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
  float back;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(back) : "f"(s));
  const float down = -s * unit;
  back *= inv;
  const Pair b2 = pair_of(back, back), d2 = pair_of(down, down);
  Pair z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[i] = f2_mul(x[i], b2);
    const Pair fine = f2_fma(f2_fma(z[i], d2, x[i]), b2, z[i]);
    if (s8 == 0x7e) {                        // elements past the largest have no remainder to speak of, or a NaN
      const float2 q = floats_of(z[i]), f = floats_of(fine);
      z[i] = pair_of(fabsf(q.x) < 8.0f ? f.x : q.x, fabsf(q.y) < 8.0f ? f.y : q.y);
    } else {
      z[i] = fine;
    }
  }
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes |= (uint32_t)__nv_cvt_float2_to_fp4x2(floats_of(z[i]), __NV_E2M1, cudaRoundNearest) << (8 * i);
  return codes;
}

template <int DT, int LANES, bool FULL, bool APPEND>   // FULL: D = 8 LANES
__global__ void __launch_bounds__(kWarps * 32, APPEND ? 8 : 7)
    heads_kernel(const __grid_constant__ HeadsArgs a, int log_parts) {
  using T = typename Elem<DT>::T;
  constexpr int kBeside = 32 / LANES;        // heads side by side in a warp
  constexpr int kHeads = 2 * kBeside;        // heads of a chunk: two steps
  constexpr int kChunkBytes = 512 * (int)sizeof(T), kRingBytes = ring_bytes(APPEND), kStages = kRingBytes / kChunkBytes;
  __shared__ __align__(128) uint8_t ring_s[kWarps][kRingBytes];
  __shared__ __align__(16) float CS[kWarps][2][LANES * 8];
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ int abort[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES, D = FULL ? 8 * LANES : a.D;
  const int64_t job = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t row = job >> log_parts;
  if (row >= a.rows) return;
  const int parts = 1 << log_parts, part = (int)(job - (row << log_parts));
  const bool live = FULL || 8 * sub < D;

  // The chunks: query heads, key heads, value heads; this warp's are part, part + parts, ...
  const int n_q = (a.Hq + kHeads - 1) / kHeads, n_k = (a.Hkv + kHeads - 1) / kHeads;
  const int chunks = n_q + (APPEND ? 2 : 1) * n_k;
  const uint32_t ring = smem_u32(ring_s[warp]), bar = smem_u32(bars[warp]);
  if (lane < kStages) mbar_init(bar + 8 * lane, 1);
  if (lane == 0) abort[warp] = 0;
  __syncwarp();
  fence_barrier_init();
  fence_proxy_async_smem();
  __syncwarp();
  const uint32_t head_bytes = D * sizeof(T);
  const uint64_t policy = policy_evict_first();
  auto issue = [&](int c, int stage) {
    const bool is_q = c < n_q, is_k = c < n_q + n_k;
    const int h0 = (is_q ? c : (is_k ? c - n_q : c - n_q - n_k)) * kHeads;
    const int n = min(kHeads, (is_q ? a.Hq : a.Hkv) - h0);
    const int64_t rs = is_q ? a.q_row : (is_k ? a.k_row : a.v_row), hs = is_q ? a.q_head : (is_k ? a.k_head : a.v_head);
    const T *p = reinterpret_cast<const T *>(is_q ? a.q : (is_k ? a.k : a.v)) + row * rs + h0 * hs;
    if (lane == 0) mbar_arrive_tx(bar + 8 * stage, n * head_bytes);
    if (hs == D) {                           // heads without gaps: one copy
      if (lane == 0) bulk_g2s(ring + stage * kChunkBytes, p, n * head_bytes, bar + 8 * stage, policy);
    } else {
      __syncwarp();
      if (lane < n) bulk_g2s(ring + stage * kChunkBytes + lane * head_bytes, p + lane * hs, head_bytes, bar + 8 * stage, policy);
    }
  };
  for (int i = 0; i < kStages && part + i * parts < chunks; ++i) issue(part + i * parts, i);

  Eight<DT> w0 = {}, w1 = {};
  if (live && a.q_weight) w0 = load8<DT>(a.q_weight, 8 * sub);
  if (live && a.k_weight) w1 = load8<DT>(a.k_weight, 8 * sub);
  // A failed step, and a row that has no place, does nothing; but no copy may be under way at the end.
  RowPlace place = {};
  const int status = status_on_entry(a.dev_status);          // looked at after the look-up, whose loads need not wait for it
  const bool found = !APPEND || find_row(a.row_off, a.kv_len, a.table, a.B, a.max_pages, a.page_size, row, lane,
                                         a.dev_status, &place);
  const int half = a.rot / 2;
  const bool turned = 8 * sub < a.rot;
  Pair c[4] = {}, s[4] = {};
  if (half && found) {
    const int64_t pos = (APPEND && !a.positions) ? place.pos : (int64_t)a.positions[row];
    float *C = CS[warp][0], *S = CS[warp][1];
    for (int i = lane; i < half; i += 32) {
      const unsigned long long turn = (unsigned long long)pos * a.turns[i];
      float sn, cs;
      sin_cos((uint32_t)(turn >> 32), &sn, &cs);
      const int d0 = a.interleaved ? 2 * i : i, d1 = a.interleaved ? 2 * i + 1 : i + half;
      C[d0] = C[d1] = cs * a.gain;
      S[d0] = -sn * a.gain;
      S[d1] = sn * a.gain;
    }
    __syncwarp();
    if (turned) {
      const ulonglong2 *cp = reinterpret_cast<const ulonglong2 *>(&C[8 * sub]);
      const ulonglong2 *sp = reinterpret_cast<const ulonglong2 *>(&S[8 * sub]);
      c[0] = cp[0].x, c[1] = cp[0].y, c[2] = cp[1].x, c[3] = cp[1].y;
      s[0] = sp[0].x, s[1] = sp[0].y, s[2] = sp[1].x, s[3] = sp[1].y;
    }
  }
  const int other = !turned ? sub : (8 * sub < half ? sub + a.rot / 16 : sub - a.rot / 16);
  const float inv_d = 1.0f / (float)D;
  const bool whole = a.rot == 8 * LANES;     // every lane's dimensions turn
  // norm (with a weight) and rotation of the heads that the warp holds
  auto turn_heads = [&](Pair (&x)[4], bool normed, const Pair (&w)[4]) {
    if (normed) {
      Pair s2 = f2_mul(x[0], x[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) s2 = f2_fma(x[e], x[e], s2);
      const float2 f = floats_of(s2);
      float ss = f.x + f.y;
#pragma unroll
      for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
      const Pair r2 = pair_of(r, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = f2_mul(f2_mul(x[e], r2), w[e]);
    }
    if (half) {
      Pair y[4];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = floats_of(x[e]);
          y[e] = pair_of(f.y, f.x);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = floats_of(x[e]);
          y[e] = pair_of(__shfl_sync(0xffffffffu, f.x, other, LANES), __shfl_sync(0xffffffffu, f.y, other, LANES));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {          // a select, not a branch that lanes take apart
        const Pair z = f2_fma(x[e], c[e], f2_mul(y[e], s[e]));
        x[e] = whole || turned ? z : x[e];
      }
    }
  };

  const bool run = !status && found && (!APPEND || place_row(a.pages, a.page_size, a.Hkv, a.dev_status, &place));
  Pair w[4];
  to_pairs<DT>(part < n_q ? w0 : w1, w);
  const int beside = lane / LANES;
  const int64_t tile_step = APPEND ? (int64_t)(a.page_size / kTileTokens) * tile_bytes(D) : 0;
  const int w16 = D / 16, at = 4 * sub, t = place.t;      // the lane's 4 bytes of a head
  T *const q_to = reinterpret_cast<T *>(a.q_out) + (row * a.Hq + beside) * D + 8 * sub;
  T *const k_to = APPEND ? nullptr : reinterpret_cast<T *>(a.k_out) + (row * a.Hkv + beside) * D + 8 * sub;
  uint8_t *const tile = APPEND ? a.cache + place.tile * tile_bytes(D) + beside * tile_step : nullptr;
  const int k_at = tile_k(D, t) + at, v_at = tile_v(D, t, at / w16) + at % w16;
  const int ks_at = tile_ks(D, t, sub >> 1), vs_at = tile_vs(D, t, sub >> 1);
  const uint8_t *const mine = ring_s[warp] + (beside * D + 8 * sub) * sizeof(T);
  int stage = 0;
  uint32_t phase = 0;
  for (int c = part; c < chunks; c += parts) {
    if (!mbar_try(bar + 8 * stage, phase) && !mbar_wait(bar + 8 * stage, phase, &abort[warp])) {
      if (lane == 0) set_status(a.dev_status, DSPARK_ERR_DEVICE_TIMEOUT);
      for (int i = 0; i < kStages && c < chunks; ++i, c += parts) {   // copies on their way get one more bounded wait
        const long long t0 = clock64();
        while (!mbar_try(bar + 8 * stage, phase) && clock64() - t0 < kTimeoutCycles / 8) {
        }
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
      return;
    }
    Pair x[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Eight<DT> v = {};
      if (live) v = *reinterpret_cast<const Eight<DT> *>(mine + stage * kChunkBytes + i * kBeside * D * sizeof(T));
      to_pairs<DT>(v, x[i]);
    }
    __syncwarp();
    if (c + kStages * parts < chunks) issue(c + kStages * parts, stage);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
    if (!run) continue;
    if (c < n_q) {
      const int h0 = c * kHeads, left = a.Hq - h0 - beside;
      turn_heads(x[0], a.q_weight != nullptr, w);
      turn_heads(x[1], a.q_weight != nullptr, w);
      T *to = q_to + h0 * D;
      if (live && left > 0) store_pairs<DT>(to, x[0]);
      if (live && left > kBeside) store_pairs<DT>(to + kBeside * D, x[1]);
      if (c + parts >= n_q) to_pairs<DT>(w1, w);           // the next chunk holds keys
      continue;
    }
    const bool is_v = c >= n_q + n_k;
    const int h0 = (is_v ? c - n_q - n_k : c - n_q) * kHeads, left = a.Hkv - h0 - beside;
    if (!is_v) {
      turn_heads(x[0], a.k_weight != nullptr, w);
      turn_heads(x[1], a.k_weight != nullptr, w);
    }
    if (!APPEND) {
      T *to = k_to + h0 * D;
      if (live && left > 0) store_pairs<DT>(to, x[0]);
      if (live && left > kBeside) store_pairs<DT>(to + kBeside * D, x[1]);
      continue;
    }
    uint8_t *to = tile + h0 * tile_step;
#pragma unroll
    for (int i = 0; i < 2; ++i, to += kBeside * tile_step) {
      uint8_t scale;
      const uint32_t codes = quantize8(x[i], is_v ? a.v_inv : a.k_inv, is_v ? a.v_unit : a.k_unit, &scale);
      if (live && left > i * kBeside) {
        *reinterpret_cast<uint32_t *>(to + (is_v ? v_at : k_at)) = codes;
        if (!(sub & 1)) to[is_v ? vs_at : ks_at] = scale;
      }
    }
  }
}

// Four e2m1 codes (the low 16 bits) as four e4m3 bytes of the same values.
__device__ __forceinline__ uint32_t e2m1_to_e4m3(uint32_t c) {
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, c & 0x7777u);
  const uint32_t sgn = ((c & 0x8u) << 4) | ((c & 0x80u) << 8) | ((c & 0x800u) << 12) | ((c & 0x8000u) << 16);
  return mag | sgn;
}

__global__ void __launch_bounds__(kWarps * 32, 16) read_kernel(const __grid_constant__ CacheReadArgs a) {
  const int status = status_on_entry(a.dev_status);
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  RowPlace p;
  if (row >= a.rows || !find_row(a.row_off, a.kv_len, a.table, a.B, a.max_pages, a.page_size, row, lane, a.dev_status, &p) ||
      !place_row(a.pages, a.page_size, a.Hkv, a.dev_status, &p) || status)
    return;
  // a lane's 4 bytes of codes are 8 elements; D/8 (a power of two) lanes take a head
  const int D = a.D, per = D / 8, w = D / 16, t = p.t, sub = lane & (per - 1), b = 4 * sub, beside = 32 / per;
  const int64_t head_bytes = (int64_t)(a.page_size / kTileTokens) * tile_bytes(D);
  const int h0 = lane / per;
  const uint8_t *tile = a.cache + p.tile * tile_bytes(D) + h0 * head_bytes;
  const int v_at = tile_v(D, t, b / w) + b % w;
  int64_t at = (row * a.Hkv + h0) * D + 8 * sub;
#pragma unroll 4
  for (int h = h0; h < a.Hkv; h += beside, tile += beside * head_bytes, at += beside * D) {
    const uint32_t k = *reinterpret_cast<const uint32_t *>(tile + tile_k(D, t) + b);
    const uint32_t v = *reinterpret_cast<const uint32_t *>(tile + v_at);
    *reinterpret_cast<uint2 *>(a.k + at) = make_uint2(e2m1_to_e4m3(k), e2m1_to_e4m3(k >> 16));
    *reinterpret_cast<uint2 *>(a.v + at) = make_uint2(e2m1_to_e4m3(v), e2m1_to_e4m3(v >> 16));
    if (!(sub & 1)) {
      a.ks[at >> 4] = tile[tile_ks(D, t, sub >> 1)];
      a.vs[at >> 4] = tile[tile_vs(D, t, sub >> 1)];
    }
  }
}

template <int DT, int LANES, bool APPEND>
cudaError_t launch_lanes(const HeadsArgs &a, cudaStream_t s) {
  // a row's heads in shares as long as the rows alone make fewer than kEnoughWarps warps
  int log_parts = 0;
  const int most = (a.Hq + (APPEND ? 2 : 1) * a.Hkv) * LANES / 64;      // chunks
  while ((a.rows << log_parts) < kEnoughWarps && 2 << log_parts <= most) ++log_parts;
  const int64_t jobs = a.rows << log_parts;
  const unsigned grid = (unsigned)((jobs + kWarps - 1) / kWarps);
  if constexpr (APPEND) {
    heads_kernel<DT, LANES, true, true><<<grid, kWarps * 32, 0, s>>>(a, log_parts);
  } else {
    if (a.D == 8 * LANES)
      heads_kernel<DT, LANES, true, false><<<grid, kWarps * 32, 0, s>>>(a, log_parts);
    else
      heads_kernel<DT, LANES, false, false><<<grid, kWarps * 32, 0, s>>>(a, log_parts);
  }
  return cudaGetLastError();
}

template <int DT, bool APPEND>
cudaError_t launch_heads(const HeadsArgs &a, cudaStream_t s) {
  if constexpr (!APPEND)                     // the cache holds heads of 64 and 128 dimensions
    if (a.D > 128) return launch_lanes<DT, 32, false>(a, s);
  return a.D <= 64 ? launch_lanes<DT, 8, APPEND>(a, s) : launch_lanes<DT, 16, APPEND>(a, s);
}

template <bool APPEND>
cudaError_t launch_heads_dt(const HeadsArgs &a, cudaStream_t s) {
  switch (a.dtype) {
    case DSPARK_BF16: return launch_heads<DSPARK_BF16, APPEND>(a, s);
    case DSPARK_F16: return launch_heads<DSPARK_F16, APPEND>(a, s);
    default: return launch_heads<DSPARK_F32, APPEND>(a, s);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const HeadsArgs &a, cudaStream_t s) { return launch_heads_dt<false>(a, s); }
cudaError_t launch_cache_append(const HeadsArgs &a, cudaStream_t s) { return launch_heads_dt<true>(a, s); }

cudaError_t launch_cache_read(const CacheReadArgs &a, cudaStream_t s) {
  read_kernel<<<(unsigned)((a.rows + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace dspark
