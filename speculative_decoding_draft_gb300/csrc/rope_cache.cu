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
// A warp takes one row, or one of `parts` equal shares of its heads, by itself: it finds the row's
// place, computes its cosines and sines once, keeps them in registers and goes over the heads with
// nothing to wait for but its loads, two of them ahead.  A lane holds 8 neighbouring dimensions of a
// head (one 16-byte load), a head takes D/8 lanes, and the partner of the half layout lies rot/16
// lanes away; with every dimension's cosine and signed sine both layouts are x C + partner S.
// Arithmetic goes in pairs of fp32 (one instruction for two).
//
// The issue slots bound it before memory does: rows spread over a CTA's threads, each finding its row
// and head by division, cost 8800 instructions for a row of 48 heads of 128 dimensions.
#include "attn.cuh"

namespace dspark {
namespace {

constexpr int kEnoughWarps = 4096;
constexpr int kWarps = 4;          // of a CTA; they share nothing

using Pair = unsigned long long;   // two fp32

__device__ __forceinline__ Pair pair_of(float lo, float hi) { return f2_pack(lo, hi); }
__device__ __forceinline__ float2 floats_of(Pair p) {
  float2 r;
  f2_unpack(p, r.x, r.y);
  return r;
}

// 8 elements as four pairs and back.
template <int DT>
__device__ __forceinline__ void to_pairs(const Eight<DT> &v, Pair (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pair_of(Elem<DT>::to(v.e[2 * i]), Elem<DT>::to(v.e[2 * i + 1]));
}
template <int DT>
__device__ __forceinline__ void store_pairs(void *base, int64_t at, const Pair (&x)[4]) {
  Eight<DT> v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = floats_of(x[i]);
    v.e[2 * i] = Elem<DT>::from(f.x);
    v.e[2 * i + 1] = Elem<DT>::from(f.y);
  }
  *reinterpret_cast<Eight<DT> *>(reinterpret_cast<typename Elem<DT>::T *>(base) + at) = v;
}
template <int DT>
__device__ __forceinline__ Eight<DT> load8(const void *base, int64_t at) {
  return *reinterpret_cast<const Eight<DT> *>(reinterpret_cast<const typename Elem<DT>::T *>(base) + at);
}

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN stays
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// Sine and cosine of an angle of turn / 2^32 turns: the nearest quarter turn by integers, the rest
// (up to pi / 4) by the Taylor series, whose first terms left out are below 2^-29 and 2^-25.
__device__ __forceinline__ void sin_cos(uint32_t turn, float *sn, float *cs) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(turn - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float y = x * x;
  float s = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(y, s, 8.3333333e-3f);
  s = fmaf(y, s, -1.6666667e-1f);
  s = fmaf(x * y, s, x);
  float c = fmaf(y, 2.4801587e-5f, -1.3888889e-3f);
  c = fmaf(y, c, 4.1666667e-2f);
  c = fmaf(y, c, -0.5f);
  c = fmaf(y, c, 1.0f);
  const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
  *sn = quarter & 2 ? -a : a;
  *cs = (quarter + 1) & 2 ? -b : b;
}

// One lane's 8 elements of a group of 16 as codes, and the group's scale.  The lane beside holds the
// others; inv is a power of two.
template <bool EXACT>
__device__ __forceinline__ uint32_t quantize8(const Pair (&x)[4], float inv, uint8_t *scale) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = floats_of(x[i]);
    top = max_nan(top, max_nan(fabsf(f.x), fabsf(f.y)));
  }
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  float sixth = top * inv;
  if (EXACT) {
    sixth = __fdiv_rn(sixth, 6.0f);
  } else {
    // Six times the border of two scales has 7 bits, so a 16-bit value's sixth is a border exactly or off
    // it by 2^-12: rounded to 21 bits the product, off by 2^-23, meets the borders without a division.
    sixth = __uint_as_float((__float_as_uint(sixth * (1.0f / 6.0f)) + 4u) & ~7u);
  }
  const __nv_fp8_storage_t s8 = __nv_cvt_float_to_fp8(sixth, __NV_SATFINITE, __NV_E4M3);
  *scale = s8;
  // 0 (nothing to keep) and NaN (nothing else to say) leave the elements 0
  if ((s8 & 0x7f) == 0 || (s8 & 0x7f) == 0x7f) return 0;
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
  Pair z[4];
  if (EXACT) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = floats_of(x[i]);
      z[i] = pair_of(__fdiv_rn(f.x * inv, s), __fdiv_rn(f.y * inv, s));
    }
  } else {
    // The quotient of a value of up to 11 bits by a scale of 4 is the border of two codes exactly or
    // off it by 2^-13 at least.  The product with the reciprocal is off by 2^-19.7 at most (up to 6.4):
    // rounded to a multiple of 2^-18 it meets the borders exactly, without a division.
    float back;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(back) : "f"(s));
    back *= inv;
    const Pair b2 = pair_of(back, back), up = pair_of(48.0f, 48.0f), down = pair_of(-48.0f, -48.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = f2_add(f2_add(f2_mul(x[i], b2), up), down);
  }
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes |= (uint32_t)__nv_cvt_float2_to_fp4x2(floats_of(z[i]), __NV_E2M1, cudaRoundNearest) << (8 * i);
  return codes;
}

template <int DT, int LANES, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32, APPEND ? 6 : 8) heads_kernel(const __grid_constant__ HeadsArgs a, int log_parts) {
  using T = typename Elem<DT>::T;
  constexpr int kBeside = 32 / LANES;        // heads side by side in a warp
  __shared__ __align__(16) float CS[kWarps][2][LANES * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES, D = a.D;
  const int64_t job = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t row = job >> log_parts;
  if (row >= a.rows) return;
  const int h0 = (int)(job - (row << log_parts)) * kBeside + lane / LANES, step = kBeside << log_parts;
  const bool live = 8 * sub < D;
  // all loads that wait for nothing, before the first wait
  const T *qp = reinterpret_cast<const T *>(a.q) + row * a.q_row + h0 * a.q_head + 8 * sub;
  const int64_t q_step = step * a.q_head;
  auto fetch = [&](const T *p, bool on) {
    Eight<DT> v = {};
    if (on) v = *reinterpret_cast<const Eight<DT> *>(p);
    return v;
  };
  Eight<DT> raw0 = fetch(qp, live && h0 < a.Hq), raw1 = fetch(qp + q_step, live && h0 + step < a.Hq);
  Eight<DT> w0 = {};
  if (live && a.q_weight) w0 = load8<DT>(a.q_weight, 8 * sub);
  if (read_status(a.dev_status)) return;
  RowPlace place = {};
  if (APPEND && !place_row(a.row_off, a.kv_len, a.table, a.B, a.max_pages, a.pages, a.page_size, a.Hkv, row, lane,
                           a.dev_status, &place))
    return;
  const int half = a.rot / 2;
  const bool turned = 8 * sub < a.rot;
  Pair c[4], s[4];
  if (half) {
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
      if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = f2_fma(x[e], c[e], f2_mul(y[e], s[e]));
      }
    }
  };

  Pair w[4];
  to_pairs<DT>(w0, w);
  const T *kp = reinterpret_cast<const T *>(a.k) + row * a.k_row + h0 * a.k_head + 8 * sub;
  const int64_t k_step = step * a.k_head;
  T *op = reinterpret_cast<T *>(a.q_out) + (row * a.Hq + h0) * D + 8 * sub;
  const int out_step = step * D;
  const int beside = lane / LANES;           // the loops run by the warp's first head, so that all lanes stay in them
  qp += 2 * q_step;
  for (int h = h0; h - beside < a.Hq; h += step, op += out_step, qp += q_step) {
    Pair x[4];
    to_pairs<DT>(raw0, x);
    raw0 = raw1;
    raw1 = fetch(qp, live && h + 2 * step < a.Hq);
    turn_heads(x, a.q_weight != nullptr, w);
    if (live && h < a.Hq) store_pairs<DT>(op, 0, x);
  }
  if (a.Hkv == 0) return;

  if (a.k_weight) {
    Eight<DT> v = {};
    if (live) v = load8<DT>(a.k_weight, 8 * sub);
    to_pairs<DT>(v, w);
  }
  raw0 = fetch(kp, live && h0 < a.Hkv), raw1 = fetch(kp + k_step, live && h0 + step < a.Hkv);
  kp += 2 * k_step;
  if (!APPEND) {
    op = reinterpret_cast<T *>(a.k_out) + (row * a.Hkv + h0) * D + 8 * sub;
    for (int h = h0; h - beside < a.Hkv; h += step, op += out_step, kp += k_step) {
      Pair x[4];
      to_pairs<DT>(raw0, x);
      raw0 = raw1;
      raw1 = fetch(kp, live && h + 2 * step < a.Hkv);
      turn_heads(x, a.k_weight != nullptr, w);
      if (live && h < a.Hkv) store_pairs<DT>(op, 0, x);
    }
    return;
  }
  const T *vp = reinterpret_cast<const T *>(a.v) + row * a.v_row + h0 * a.v_head + 8 * sub;
  const int64_t v_step = step * a.v_head;
  Eight<DT> v0 = fetch(vp, live && h0 < a.Hkv), v1 = fetch(vp + v_step, live && h0 + step < a.Hkv);
  vp += 2 * v_step;
  const int64_t head_bytes = (int64_t)(a.page_size / kTileTokens) * tile_bytes(D), tile_step = step * head_bytes;
  const int w16 = D / 16, at = 4 * sub, t = place.t;      // the lane's 4 bytes of a head
  uint8_t *tile = a.cache + place.tile * tile_bytes(D) + h0 * head_bytes;
  const int k_at = tile_k(D, t) + at, v_at = tile_v(D, t, at / w16) + at % w16;
  const int ks_at = tile_ks(D, t, sub >> 1), vs_at = tile_vs(D, t, sub >> 1);
  for (int h = h0; h - beside < a.Hkv; h += step, kp += k_step, vp += v_step, tile += tile_step) {
    Pair x[4];
    uint8_t scale;
    to_pairs<DT>(raw0, x);
    raw0 = raw1;
    raw1 = fetch(kp, live && h + 2 * step < a.Hkv);
    turn_heads(x, a.k_weight != nullptr, w);
    uint32_t codes = quantize8<DT == DSPARK_F32>(x, a.k_inv, &scale);
    if (live && h < a.Hkv) {
      *reinterpret_cast<uint32_t *>(tile + k_at) = codes;
      if (!(sub & 1)) tile[ks_at] = scale;
    }
    to_pairs<DT>(v0, x);
    v0 = v1;
    v1 = fetch(vp, live && h + 2 * step < a.Hkv);
    codes = quantize8<DT == DSPARK_F32>(x, a.v_inv, &scale);
    if (live && h < a.Hkv) {
      *reinterpret_cast<uint32_t *>(tile + v_at) = codes;
      if (!(sub & 1)) tile[vs_at] = scale;
    }
  }
}

// Four e2m1 codes (the low 16 bits) as four e4m3 bytes of the same values.
__device__ __forceinline__ uint32_t e2m1_to_e4m3(uint32_t c) {
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, c & 0x7777u);
  const uint32_t sgn = ((c & 0x8u) << 4) | ((c & 0x80u) << 8) | ((c & 0x800u) << 12) | ((c & 0x8000u) << 16);
  return mag | sgn;
}

__global__ void __launch_bounds__(kWarps * 32) read_kernel(const __grid_constant__ CacheReadArgs a) {
  if (read_status(a.dev_status)) return;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  RowPlace p;
  if (row >= a.rows || !place_row(a.row_off, a.kv_len, a.table, a.B, a.max_pages, a.pages, a.page_size, a.Hkv, row, lane,
                                  a.dev_status, &p))
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
  // a row's heads in shares as long as the rows alone leave the SMs without work: 24 warps on each of
  // 152 and several rounds of them
  int log_parts = 0;
  const int most = ((a.Hq > a.Hkv ? a.Hq : a.Hkv) * LANES + 31) / 32;
  while ((a.rows << log_parts) < kEnoughWarps && 2 << log_parts <= most) ++log_parts;
  const int64_t jobs = a.rows << log_parts;
  heads_kernel<DT, LANES, APPEND><<<(unsigned)((jobs + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a, log_parts);
  return cudaGetLastError();
}

template <int DT, bool APPEND>
cudaError_t launch_heads(const HeadsArgs &a, cudaStream_t s) {
  if (a.D <= 64) return launch_lanes<DT, 8, APPEND>(a, s);
  if (a.D <= 128) return launch_lanes<DT, 16, APPEND>(a, s);
  return launch_lanes<DT, 32, APPEND>(a, s);
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
