// Device code that the kernels on query and key heads share: 8 neighbouring dimensions of a lane as pairs of fp32,
// and the angles of the rotation.
#pragma once

#include "attn.cuh"

namespace dspark {

using Pair = unsigned long long;   // two fp32

__device__ __forceinline__ Pair pair_of(float lo, float hi) { return f2_pack(lo, hi); }
__device__ __forceinline__ float2 floats_of(Pair p) {
  float2 r;
  f2_unpack(p, r.x, r.y);
  return r;
}

// 8 elements as four pairs and back, two elements with one conversion.
template <int DT>
__device__ __forceinline__ void to_pairs(const Eight<DT> &v, Pair (&x)[4]) {
  const uint32_t *u = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == DSPARK_BF16) {
      x[i] = pair_of(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    } else if constexpr (DT == DSPARK_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
      x[i] = pair_of(f.x, f.y);
    } else {
      x[i] = pair_of(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
    }
  }
}
template <int DT>
__device__ __forceinline__ void store_pairs(void *to, const Pair (&x)[4]) {
  if constexpr (DT == DSPARK_F32) {
    ulonglong2 *p = reinterpret_cast<ulonglong2 *>(to);
    p[0] = make_ulonglong2(x[0], x[1]);
    p[1] = make_ulonglong2(x[2], x[3]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = floats_of(x[i]);
      if constexpr (DT == DSPARK_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    *reinterpret_cast<uint4 *>(to) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}
template <int DT>
__device__ __forceinline__ Eight<DT> load8(const void *base, int64_t at) {
  return *reinterpret_cast<const Eight<DT> *>(reinterpret_cast<const typename Elem<DT>::T *>(base) + at);
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

}  // namespace dspark
