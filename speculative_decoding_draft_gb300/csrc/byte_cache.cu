// The append of keys and values to the paged cache in 8 bits, with norm and rotation of queries and keys on the way,
// and the cache's read-back as values.
//
//   y = x rsqrt(mean(x^2) + eps) w, rotated          (queries and keys; as norm_rope)
//   e = the smallest with 448 2^e >= max |y| over the finite y of a block, element = e4m3(y 2^-e)
// for the 16 tokens of a block of one head, keys and values apart.  A scale is a power of two, so that a block whose
// scale rises, because a later token is louder, keeps its elements but for those that fall below the normal numbers
// of e4m3: moving them is a change of exponents.
//
// A run is the rows of one call that fall into one block: up to 16.  A CTA takes the runs that begin in a window of rows
// (its heads shared out over `parts` CTAs where rows are few): 8 warps make the angles of the run's rows once for
// all heads, then a warp takes the keys or the values of one head, twice over the rows of the run, since the scale is
// known only when all of them are (held in registers between the two, 16 rows took 128 registers a thread, and
// half the warps on an SM); queries go row by row.  A lane holds 8 neighbouring dimensions.
//
// Measured (one GB300): 9216 rows of 2048 requests with 32 query and 8 key/value heads of 128 dimensions 111 us (30 us at
// the memory's rate), bound by issue slots (52 % busy) and by a run's steps that follow one another (look-up, angles, two
// sweeps, queries); their read-back with the rest of the touched blocks 35 us (22), bound by the look-up's latency.
//
// All arithmetic is in fp32; queries are rounded once to their type, keys and values once to 8 bits, and once more
// where a block's scale rises behind them.
#include "heads.cuh"

namespace dspark {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kELow = -32, kEHigh = 31;              // exponents of a block's scale

// The exponent of the smallest scale whose largest element reaches the magnitude with these bits.
__device__ __forceinline__ int exponent_for(uint32_t top) {
  return min(max((int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u), kELow), kEHigh);
}
__device__ __forceinline__ int exponent_held(uint8_t b) { return min(max((int)b - 127, kELow), kEHigh); }
__device__ __forceinline__ float two_to(int e) { return __int_as_float((127 + e) << 23); }

// 8 values as e4m3, to nearest, ties to even; infinities become the largest, a NaN stays one.
__device__ __forceinline__ uint2 elements(const Pair (&x)[4], float unit) {
  uint32_t h[4];
  const Pair u2 = pair_of(unit, unit);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __nv_cvt_float2_to_fp8x2(floats_of(f2_mul(x[i], u2)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// The element's place in its token: 16-byte pieces lie in the order that the tensor cores' swizzle reads.
template <int D>
__device__ __forceinline__ int piece_at(int t, int c) {
  return D == 128 ? c ^ (t & 7) : c ^ ((t >> 1) & 3);
}

template <int DT>
__device__ __forceinline__ Eight<DT> load8_once(const void *p) {
  Eight<DT> v;
  const uint4 *s = reinterpret_cast<const uint4 *>(p);
  uint4 *d = reinterpret_cast<uint4 *>(&v);
#pragma unroll
  for (int i = 0; i < (int)sizeof(v) / 16; ++i) d[i] = __ldcs(s + i);
  return v;
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 3)
    append_kernel(const __grid_constant__ ByteHeadsArgs a, int window, int parts) {
  using T = typename Elem<DT>::T;
  constexpr int LANES = D / 8, kBeside = 32 / LANES, kAhead = DT == DSPARK_F32 ? 2 : 4;
  __shared__ __align__(16) float C[kTileTokens][D], S[kTileTokens][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES, beside = lane / LANES;
  const int64_t first = blockIdx.x / (unsigned)parts * (int64_t)window;
  const int part = (int)(blockIdx.x % (unsigned)parts);
  const int q0 = a.Hq * part / parts, nq = a.Hq * (part + 1) / parts - q0;
  const int h0 = a.Hkv * part / parts, nkv = a.Hkv * (part + 1) / parts - h0;
  // (the word may change while the CTA's threads read it: they leave together or not at all)
  if (__syncthreads_or(status_on_entry(a.dev_status))) return;

  // Runs begin where a request does and at every block's first token.
  const int64_t all = a.row_off[a.B];
  int64_t row = first, r = request_of_row(a.row_off, a.B, row, lane);
  const int64_t until = min(min(first + window, a.rows), all);
  const int half = a.rot / 2;
  const bool turned = 8 * sub < a.rot, all_turn = a.rot == D;
  const int other = !turned ? sub : (8 * sub < half ? sub + a.rot / 16 : sub - a.rot / 16);
  const float inv_d = 1.0f / (float)D;
  Eight<DT> w0 = {}, w1 = {};
  if (a.q_weight) w0 = load8<DT>(a.q_weight, 8 * sub);
  if (a.k_weight) w1 = load8<DT>(a.k_weight, 8 * sub);

  // norm (with a weight) and rotation of a row's 8 dimensions, the row's place in the run being i
  auto turn = [&](Pair (&x)[4], bool normed, const Eight<DT> &weight, int i) {
    if (normed) {
      Pair s2 = f2_mul(x[0], x[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) s2 = f2_fma(x[e], x[e], s2);
      const float2 f = floats_of(s2);
      float ss = f.x + f.y;
#pragma unroll
      for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
      const Pair i2 = pair_of(inv, inv);
      Pair w[4];
      to_pairs<DT>(weight, w);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = f2_mul(f2_mul(x[e], i2), w[e]);
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
      const ulonglong2 *cp = reinterpret_cast<const ulonglong2 *>(&C[i][8 * sub]);
      const ulonglong2 *sp = reinterpret_cast<const ulonglong2 *>(&S[i][8 * sub]);
      const ulonglong2 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
      const Pair c[4] = {c0.x, c0.y, c1.x, c1.y}, s[4] = {s0.x, s0.y, s1.x, s1.y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const Pair z = f2_fma(x[e], c[e], f2_mul(y[e], s[e]));
        x[e] = all_turn || turned ? z : x[e];
      }
    }
  };

  while (row < until) {
    // the request of the row (empty ones are passed over) and the row's place
    int64_t b0 = a.row_off[r], b1 = a.row_off[r + 1];
    while (b1 <= row && r + 1 < a.B) {
      ++r;
      b0 = b1;
      b1 = a.row_off[r + 1];
    }
    if (row < b0 || row >= b1 || b1 > a.rows) {
      if (threadIdx.x == 0) set_status(a.dev_status, DSPARK_ERR_OFFSETS);
      return;
    }
    const int64_t pos = (int64_t)a.kv_len[r] - b1 + row;
    if (pos - (row - b0) < 0 || pos + (b1 - 1 - row) >= a.max_pages * a.page_size) {
      if (threadIdx.x == 0) set_status(a.dev_status, DSPARK_ERR_LENGTHS);
      row = b1;
      continue;
    }
    const int t0 = (int)(pos % kTileTokens);
    const int len = (int)min(b1 - row, (int64_t)(kTileTokens - t0));
    if (t0 && row > b0) {                              // this run began in an earlier window
      row += len;
      continue;
    }
    const uint32_t tile = (uint32_t)pos / kTileTokens, per = (uint32_t)a.page_size / kTileTokens, at = tile / per;
    const int32_t page = a.table[r * a.max_pages + at];
    if (page < 0 || page >= a.pages) {
      if (threadIdx.x == 0) set_status(a.dev_status, DSPARK_ERR_PAGES);
      row += len;
      continue;
    }
    const int in_page = (int)(tile - at * per);        // the block in its page

    if (half) {                                        // the angles of the run's rows
      __syncthreads();                                 // (no one is at the last run's any more)
      for (int i = threadIdx.x; i < len * half; i += kThreads) {
        const int j = i / half, p = i - j * half;
        const int64_t where = a.positions ? (int64_t)a.positions[row + j] : pos + j;
        const unsigned long long turns = (unsigned long long)where * a.turns[p];
        float sn, cs;
        sin_cos((uint32_t)(turns >> 32), &sn, &cs);
        const int d0 = a.interleaved ? 2 * p : p, d1 = a.interleaved ? 2 * p + 1 : p + half;
        C[j][d0] = C[j][d1] = cs * a.gain;
        S[j][d0] = -sn * a.gain;
        S[j][d1] = sn * a.gain;
      }
      __syncthreads();
    }

    // keys and values: a warp has one kind of one head
    for (int u = warp; u < 2 * nkv; u += kWarps) {
      const int h = h0 + (u >> 1), kind = u & 1;
      const T *src = reinterpret_cast<const T *>(kind ? a.v : a.k) + row * (kind ? a.v_row : a.k_row) + h * (kind ? a.v_head : a.k_head) + 8 * sub;
      const int64_t src_row = kind ? a.v_row : a.k_row;
      const int64_t block = ((int64_t)page * a.Hkv + h) * 2 + kind;
      uint8_t *scale_at = a.scales + block * per + in_page;
      uint8_t *data = a.data + (block * a.page_size + in_page * kTileTokens) * D;
      const int held = t0 ? exponent_held(*scale_at) : kELow;
      // twice over the rows: for the largest magnitude, then for the elements (what is read again lies in the caches)
      auto sweep = [&](auto &&use) {
#pragma unroll 1
        for (int p0 = 0; p0 < len; p0 += kAhead * kBeside) {
          Eight<DT> in[kAhead];
#pragma unroll
          for (int p = 0; p < kAhead; ++p) {
            const int j = p0 + p * kBeside + beside;
            in[p] = j < len ? load8<DT>(src, j * src_row) : Eight<DT>{};
          }
#pragma unroll
          for (int p = 0; p < kAhead; ++p) {
            if (p0 + p * kBeside >= len) break;
            const int j = p0 + p * kBeside + beside;
            Pair x[4];
            to_pairs<DT>(in[p], x);
            if (!kind) turn(x, a.k_weight != nullptr, w1, min(j, len - 1));
            if (j < len) use(x, j);
          }
        }
      };
      float top = 0.0f;
      sweep([&](const Pair (&x)[4], int) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = floats_of(x[e]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));             // a NaN counts nothing
        }
      });
      uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      if (bits >= 0x7f800000u) {                                                  // infinities count nothing either
        top = 0.0f;
        sweep([&](const Pair (&x)[4], int) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = floats_of(x[e]);
            if (fabsf(f.x) < INFINITY) top = fmaxf(top, fabsf(f.x));
            if (fabsf(f.y) < INFINITY) top = fmaxf(top, fabsf(f.y));
          }
        });
        bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      }
      const int e = max(held, exponent_for(bits));
      const float unit = two_to(-e);
      sweep([&](const Pair (&x)[4], int j) {
        const int t = t0 + j;
        *reinterpret_cast<uint2 *>(data + t * D + piece_at<D>(t, sub >> 1) * 16 + (sub & 1) * 8) = elements(x, unit);
      });
      if (t0 && e > held) {                            // what the block holds already, on the new scale
        const float down = two_to(held - e);
        for (int i = lane; i < t0 * (D / 8); i += 32) {
          uint2 *at8 = reinterpret_cast<uint2 *>(data) + i;
          const uint2 was = *at8;
          Pair y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w = k < 2 ? was.x : was.y;
            const __half2_raw two = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (k & 1))), __NV_E4M3);
            const float2 f = __half22float2(__half2(two));
            y[k] = pair_of(f.x, f.y);
          }
          *at8 = elements(y, down);
        }
      }
      if (lane == 0) *scale_at = (uint8_t)(e + 127);
    }

    // queries: a row's head takes LANES lanes, four steps under way
    const int units = len * nq;
    const uint32_t inv_nq = nq > 1 ? 0xffffffffu / nq + 1 : 0;   // u / nq = high word of the product, u nq being below 2^32
    for (int u0 = warp * 4 * kBeside; u0 < units; u0 += kWarps * 4 * kBeside) {
      Eight<DT> in[4];
      int j[4], h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int u = min(u0 + k * kBeside + beside, units - 1);
        j[k] = nq > 1 ? (int)__umulhi((uint32_t)u, inv_nq) : u;
        h[k] = q0 + u - j[k] * nq;
        in[k] = load8_once<DT>(reinterpret_cast<const T *>(a.q) + (row + j[k]) * a.q_row + h[k] * a.q_head + 8 * sub);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (u0 + k * kBeside >= units) break;
        Pair x[4];
        to_pairs<DT>(in[k], x);
        turn(x, a.q_weight != nullptr, w0, j[k]);
        if (u0 + k * kBeside + beside < units)
          store_pairs<DT>(reinterpret_cast<T *>(a.q_out) + ((row + j[k]) * a.Hq + h[k]) * D + 8 * sub, x);
      }
    }
    row += len;
  }
}

// A warp takes a row, or one of `parts` shares of its heads: D/16 lanes a head's keys or values, 16 elements a lane.
template <int DT, int D>
__global__ void __launch_bounds__(128) read_kernel(const __grid_constant__ ByteReadArgs a, int parts) {
  using T = typename Elem<DT>::T;
  constexpr int kLanes = D / 16, kBeside = 32 / kLanes;
  const int status = status_on_entry(a.dev_status);
  const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), row = job / parts;
  const int lane = threadIdx.x & 31, part = (int)(job - row * parts);
  RowPlace p;
  if (row >= a.rows || !find_row(a.row_off, a.kv_len, a.table, a.B, a.max_pages, a.page_size, row, lane, a.dev_status, &p) ||
      !place_row(a.pages, a.page_size, a.Hkv, a.dev_status, &p) || status)
    return;
  const int per = a.page_size / kTileTokens, c = lane % kLanes, in_page = p.in_page * kTileTokens + p.t;
  const int u0 = 2 * a.Hkv * part / parts, u1 = 2 * a.Hkv * (part + 1) / parts;   // kinds of heads: head u / 2, kind u % 2
#pragma unroll 4
  for (int u = u0 + lane / kLanes; u < u1; u += kBeside) {
    const int64_t block = ((int64_t)p.page * a.Hkv + (u >> 1)) * 2 + (u & 1);
    const uint4 x = *reinterpret_cast<const uint4 *>(a.data + (block * a.page_size + in_page) * D + piece_at<D>(p.t, c) * 16);
    const float unit = two_to(exponent_held(a.scales[block * per + p.in_page]));
    const Pair u2 = pair_of(unit, unit);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    T *to = reinterpret_cast<T *>((u & 1) ? a.v : a.k) + (row * a.Hkv + (u >> 1)) * D + 16 * c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Pair y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2_raw two = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[2 * i + k / 2] >> (16 * (k & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(two));
        y[k] = f2_mul(pair_of(f.x, f.y), u2);
      }
      store_pairs<DT>(to + 8 * i, y);
    }
  }
}

template <int DT, int D>
cudaError_t append(const ByteHeadsArgs &a, cudaStream_t s, int sms) {
  // windows of rows until two waves of CTAs are full, then heads shared out where rows are few
  const int64_t enough = 6 * (int64_t)sms;          // (12, 24 and 48: 9216 rows 149, 155 and 168 us, 8190 rows 31, 37 and 48 against 29)
  int window = 16, parts = 1;
  while (window > 1 && (a.rows + window - 1) / window < enough) window /= 2;
  const int64_t windows = (a.rows + window - 1) / window;
  while (2 * parts <= a.Hkv && windows * parts < enough / 2) parts *= 2;
  append_kernel<DT, D><<<(unsigned)(windows * parts), kThreads, 0, s>>>(a, window, parts);
  return cudaGetLastError();
}
template <int DT, int D>
cudaError_t read(const ByteReadArgs &a, cudaStream_t s, int sms) {
  int parts = 1;
  while (2 * parts <= a.Hkv && a.rows * parts < 16 * (int64_t)sms) parts *= 2;
  read_kernel<DT, D><<<(unsigned)((a.rows * parts + 3) / 4), 128, 0, s>>>(a, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_byte_append(const ByteHeadsArgs &a, cudaStream_t s, int sms) {
  switch (a.dtype) {
    case DSPARK_BF16: return a.D == 128 ? append<DSPARK_BF16, 128>(a, s, sms) : append<DSPARK_BF16, 64>(a, s, sms);
    case DSPARK_F16: return a.D == 128 ? append<DSPARK_F16, 128>(a, s, sms) : append<DSPARK_F16, 64>(a, s, sms);
    default: return a.D == 128 ? append<DSPARK_F32, 128>(a, s, sms) : append<DSPARK_F32, 64>(a, s, sms);
  }
}

cudaError_t launch_byte_read(const ByteReadArgs &a, cudaStream_t s, int sms) {
  switch (a.dtype) {
    case DSPARK_BF16: return a.D == 128 ? read<DSPARK_BF16, 128>(a, s, sms) : read<DSPARK_BF16, 64>(a, s, sms);
    case DSPARK_F16: return a.D == 128 ? read<DSPARK_F16, 128>(a, s, sms) : read<DSPARK_F16, 64>(a, s, sms);
    default: return a.D == 128 ? read<DSPARK_F32, 128>(a, s, sms) : read<DSPARK_F32, 64>(a, s, sms);
  }
}

}  // namespace dspark
