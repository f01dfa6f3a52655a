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
// One CTA of 256 threads takes one row with all its heads: the row's cosines and sines are computed
// once and shared by every head.  A thread holds 8 neighbouring dimensions (one 16-byte load), a
// head takes D/8 lanes, and the partner of the half layout lies rot/16 lanes away.
#include "attn.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;

template <int DT>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&x)[8]) {
  using T = typename Elem<DT>::T;
  const Eight<DT> v = *reinterpret_cast<const Eight<DT> *>(reinterpret_cast<const T *>(base) + at);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = Elem<DT>::to(v.e[i]);
}

template <int DT>
__device__ __forceinline__ void store8(void *base, int64_t at, const float (&x)[8]) {
  using T = typename Elem<DT>::T;
  Eight<DT> v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v.e[i] = Elem<DT>::from(x[i]);
  *reinterpret_cast<Eight<DT> *>(reinterpret_cast<T *>(base) + at) = v;
}

// Norm and rotation of the 8 dimensions from 8 * sub of a head that the LANES lanes around hold.
template <int LANES>
__device__ __forceinline__ void head_norm_rope(float (&x)[8], int sub, int D, const float *w, float eps, int rot,
                                               bool interleaved, const float *cosv, const float *sinv) {
  if (w) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m, LANES);
    const float r = rsqrtf(ss / (float)D + eps);
    if (8 * sub < D) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[8 * sub + i];
    }
  }
  if (rot == 0) return;
  if (interleaved) {
    if (8 * sub < rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = cosv[4 * sub + i], s = sinv[4 * sub + i], a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * c - b * s;
        x[2 * i + 1] = b * c + a * s;
      }
    }
  } else {
    const int step = rot / 16;                       // lanes that half of the rotated part takes
    const bool first = sub < step;
    const int other = first ? sub + step : sub - step;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], other < 0 ? 0 : other, LANES);
    if (8 * sub < rot) {
      const int at = 8 * (first ? sub : other);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = cosv[at + i], s = first ? -sinv[at + i] : sinv[at + i];
        x[i] = fmaf(x[i], c, y[i] * s);
      }
    }
  }
}

// One lane's 8 elements of a group of 16 as codes, and the group's scale.
__device__ __forceinline__ uint32_t quantize8(const float (&x)[8], float inv, uint8_t *scale) {
  float y[8];
  uint32_t top = 0;      // largest magnitude by bits: a NaN counts above all
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = x[i] * inv;
    top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const __nv_fp8_storage_t s8 = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(top), 6.0f), __NV_SATFINITE, __NV_E4M3);
  *scale = s8;
  // 0 (nothing to keep) and NaN (nothing else to say) leave the elements 0
  if ((s8 & 0x7f) == 0 || (s8 & 0x7f) == 0x7f) return 0;
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)));
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the quotient of a 16-bit value can lie on the border of two codes: divided exactly, not by a reciprocal
    const float2 z = make_float2(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s));
    codes |= (uint32_t)__nv_cvt_float2_to_fp4x2(z, __NV_E2M1, cudaRoundNearest) << (8 * i);
  }
  return codes;
}

struct RowShared {
  float cosv[128], sinv[128], qw[256], kw[256];
  RowPlace place;
  int skip;
};

template <int DT, int LANES, bool APPEND>
__global__ void __launch_bounds__(kThreads) heads_kernel(const __grid_constant__ HeadsArgs a) {
  __shared__ RowShared sh;
  if (read_status(a.dev_status)) return;
  const int tid = threadIdx.x, lane = tid & 31, sub = tid % LANES;
  const int64_t row = blockIdx.x;
  for (int i = tid; i < a.D; i += kThreads) {
    using T = typename Elem<DT>::T;
    if (a.q_weight) sh.qw[i] = Elem<DT>::to(reinterpret_cast<const T *>(a.q_weight)[i]);
    if (a.k_weight) sh.kw[i] = Elem<DT>::to(reinterpret_cast<const T *>(a.k_weight)[i]);
  }
  if (APPEND) {
    if (tid < 32) {
      RowPlace p;
      const bool ok = place_row(a.row_off, a.kv_len, a.table, a.B, a.max_pages, a.pages, a.page_size, a.Hkv, row, lane,
                                a.dev_status, &p);
      if (lane == 0) {
        sh.skip = !ok;
        sh.place = p;
      }
    }
    __syncthreads();
    if (sh.skip) return;
  }
  const int half = a.rot / 2;
  if (tid < half) {
    const int64_t pos = (APPEND && !a.positions) ? sh.place.pos : (int64_t)a.positions[row];
    const unsigned long long turn = (unsigned long long)pos * a.turns[tid];
    // the top 32 bits as a signed number of half turns / 2^31
    const float x = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    sh.cosv[tid] = c * a.gain;
    sh.sinv[tid] = s * a.gain;
  }
  __syncthreads();
  const int D = a.D, heads = a.Hq + a.Hkv, units = APPEND ? heads + a.Hkv : heads;
  const bool live = 8 * sub < D;
  for (int u0 = 0; u0 < units; u0 += kThreads / LANES) {
    const int u = u0 + tid / LANES;
    const bool on = live && u < units;
    const bool is_q = u < a.Hq, is_v = u >= heads;
    const int h = is_q ? u : (is_v ? u - heads : u - a.Hq);
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (on) {
      const void *base = is_q ? a.q : (is_v ? a.v : a.k);
      const int64_t at = (is_q ? row * a.q_row + h * a.q_head
                               : (is_v ? row * a.v_row + h * a.v_head : row * a.k_row + h * a.k_head)) + 8 * sub;
      load8<DT>(base, at, x);
    }
    // lanes without a head take part in the shuffles
    const float *w = is_q ? (a.q_weight ? sh.qw : nullptr) : (a.k_weight ? sh.kw : nullptr);
    const bool any_w = a.q_weight || a.k_weight;
    if (any_w || half) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i];
      // a warp may hold query and key heads together, and only one of them normed
      if (any_w) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m, LANES);
        if (w && live) {
          const float r = rsqrtf(ss / (float)D + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] * r * w[8 * sub + i];
        }
      }
      head_norm_rope<LANES>(y, sub, D, nullptr, 0.0f, a.rot, a.interleaved, sh.cosv, sh.sinv);
      if (!is_v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = y[i];
      }
    }
    if (!APPEND) {
      if (on) store8<DT>(is_q ? a.q_out : a.k_out, (row * (is_q ? a.Hq : a.Hkv) + h) * D + 8 * sub, x);
      continue;
    }
    uint8_t scale;
    const uint32_t codes = quantize8(x, is_v ? a.v_inv : a.k_inv, &scale);
    if (!on) continue;
    if (is_q) {
      store8<DT>(a.q_out, (row * a.Hq + h) * D + 8 * sub, x);
      continue;
    }
    const int t = sh.place.t;
    uint8_t *tile = a.cache + (sh.place.tile + (int64_t)h * (a.page_size / kTileTokens)) * tile_bytes(D);
    if (is_v) {
      const int w16 = D / 16, b = 4 * sub;           // the lane's 4 bytes of the value
      *reinterpret_cast<uint32_t *>(tile + tile_v(D, t, b / w16) + b % w16) = codes;
      if (!(sub & 1)) tile[tile_vs(D, t, sub >> 1)] = scale;
    } else {
      *reinterpret_cast<uint32_t *>(tile + tile_k(D, t) + 4 * sub) = codes;
      if (!(sub & 1)) tile[tile_ks(D, t, sub >> 1)] = scale;
    }
  }
}

// Four e2m1 codes (the low 16 bits) as four e4m3 bytes of the same values.
__device__ __forceinline__ uint32_t e2m1_to_e4m3(uint32_t c) {
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, c & 0x7777u);
  const uint32_t sgn = ((c & 0x8u) << 4) | ((c & 0x80u) << 8) | ((c & 0x800u) << 12) | ((c & 0x8000u) << 16);
  return mag | sgn;
}

__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ CacheReadArgs a) {
  __shared__ RowPlace place;
  __shared__ int skip;
  if (read_status(a.dev_status)) return;
  const int64_t row = blockIdx.x;
  if (threadIdx.x < 32) {
    RowPlace p;
    const bool ok = place_row(a.row_off, a.kv_len, a.table, a.B, a.max_pages, a.pages, a.page_size, a.Hkv, row,
                              threadIdx.x, a.dev_status, &p);
    if (threadIdx.x == 0) {
      skip = !ok;
      place = p;
    }
  }
  __syncthreads();
  if (skip) return;
  const int D = a.D, per = D / 8, w = D / 16, t = place.t;
  for (int i = threadIdx.x; i < 2 * a.Hkv * per; i += kThreads) {
    const bool is_v = i >= a.Hkv * per;
    const int h = (is_v ? i - a.Hkv * per : i) / per, sub = i % per, b = 4 * sub;
    const uint8_t *tile = a.cache + (place.tile + (int64_t)h * (a.page_size / kTileTokens)) * tile_bytes(D);
    const uint32_t c = *reinterpret_cast<const uint32_t *>(is_v ? tile + tile_v(D, t, b / w) + b % w
                                                                : tile + tile_k(D, t) + b);
    const int64_t at = (row * a.Hkv + h) * D + 8 * sub;
    *reinterpret_cast<uint2 *>((is_v ? a.v : a.k) + at) = make_uint2(e2m1_to_e4m3(c), e2m1_to_e4m3(c >> 16));
    if (!(sub & 1))
      (is_v ? a.vs : a.ks)[(row * a.Hkv + h) * w + (sub >> 1)] = is_v ? tile[tile_vs(D, t, sub >> 1)]
                                                                        : tile[tile_ks(D, t, sub >> 1)];
  }
}

template <int DT, bool APPEND>
cudaError_t launch_heads(const HeadsArgs &a, cudaStream_t s) {
  const dim3 grid((unsigned)a.rows);
  if (a.D <= 64)
    heads_kernel<DT, 8, APPEND><<<grid, kThreads, 0, s>>>(a);
  else if (a.D <= 128)
    heads_kernel<DT, 16, APPEND><<<grid, kThreads, 0, s>>>(a);
  else
    heads_kernel<DT, 32, APPEND><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
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
  read_kernel<<<(unsigned)a.rows, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace dspark
