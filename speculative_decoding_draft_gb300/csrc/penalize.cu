// Penalties for repeated tokens, biases and grammar masks on the logits of ragged rows.
//
// Row i = row_off[r] + j of request r, token v, with n = how often v is among the request's output
// (history from prompt_len on) and the j draft tokens before the row, s = v is in the prompt:
//   z = logit;  if (n > 0 or s) z = z > 0 ? z / repetition : z * repetition
//   z -= presence [n > 0] + frequency n;  z += the request's biases of v;  -inf where the mask bit is 0
// in fp32, rounded once to the logits' type.
//
// Bound by memory: a row is read and written once.  One CTA takes one slice of the vocabulary for one
// request and all of its rows, so the history is read once a slice and not once a row.  It counts the
// history's tokens of its slice in shared memory with integer atomics (their order changes nothing)
// and lists every token that it may have to change (history, draft tokens, biases).  Then it goes over
// the rows twice: all of the slice, 16 bytes at a time, with the mask alone; and the few listed
// tokens, in what the first pass wrote.  (Changing them on the way, piece by piece, made the kernel
// large and divergent: 260 us where this takes NNN for 288 rows of 151936.)  In place and without
// a mask the first pass has nothing to do.
#include "attn.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                    // 16-byte pieces in flight per thread
constexpr int64_t kMaxRequestRows = 1 << 20;   // its pieces are counted in 32 bits
constexpr uint32_t kInPrompt = 0x80000000u;   // a count's top bit

struct Bias {
  int32_t at;
  float sum;
};

template <int DT, bool MASK>
__global__ void __launch_bounds__(kThreads) penalize_kernel(const __grid_constant__ PenalizeArgs a, int slice) {
  using T = typename Elem<DT>::T;
  constexpr int N = 16 / sizeof(T);           // elements of a piece
  constexpr uint32_t kAll = (1u << N) - 1;
  extern __shared__ uint32_t counts[];        // [slice]
  uint32_t *map = counts + slice;             // [slice / 32]: listed tokens
  Bias *biases = reinterpret_cast<Bias *>(map + slice / 32);                                     // [bias slots]
  uint16_t *list = reinterpret_cast<uint16_t *>(biases + (a.bias_cap < slice ? a.bias_cap : slice));   // [slice]
  __shared__ int n_list, n_bias;
  const int tid = threadIdx.x;
  const int slices = (int)((a.V + slice - 1) / slice);
  const int64_t r = blockIdx.x / slices, v0 = (int64_t)(blockIdx.x - r * slices) * slice;
  const int width = (int)(a.V - v0 < slice ? a.V - v0 : slice);
  const int status = read_status(a.dev_status);
  const int64_t first = a.row_off[r], end = a.row_off[r + 1];
  const int64_t n_hist = a.hist_len[r], n_prompt = a.prompt_len[r];
  const float rep = a.repetition[r], pre = a.presence[r], fre = a.frequency[r];
  for (int i = tid; i < (slice + slice / 32) / 4; i += kThreads) reinterpret_cast<uint4 *>(counts)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) n_list = n_bias = 0;
  if (status) return;
  if (first < 0 || end < first || end > a.rows || end - first > kMaxRequestRows ||
      (a.draft_tok && end - first > a.draft_cap + 1)) {
    if (tid == 0) set_status(a.dev_status, DSPARK_ERR_OFFSETS);
    return;
  }
  if (n_hist < 0 || n_hist > a.hist_cap || n_prompt < 0 || n_prompt > n_hist) {
    if (tid == 0) set_status(a.dev_status, DSPARK_ERR_LENGTHS);
    return;
  }
  if (end == first) return;
  __syncthreads();

  // what the slice's tokens have against them
  const int32_t *hist = a.hist + r * a.hist_cap;
  const int32_t *draft = a.draft_tok ? a.draft_tok + r * a.draft_cap : nullptr;
  auto mark = [&](int at) {
    const uint32_t bit = 1u << (at & 31);
    if (!(atomicOr(&map[at >> 5], bit) & bit)) list[atomicAdd(&n_list, 1)] = (uint16_t)at;
  };
  auto count = [&](int64_t i, int32_t tok) {
    if (tok < 0 || tok >= a.V) {
      set_status(a.dev_status, DSPARK_ERR_TOKEN_RANGE);
    } else if (tok >= v0 && tok < v0 + width) {
      const int at = (int)(tok - v0);
      if (i < n_prompt)
        atomicOr(&counts[at], kInPrompt);
      else
        atomicAdd(&counts[at], 1u);
      mark(at);
    }
  };
  for (int64_t i = tid; i < n_hist; i += 4 * kThreads) {
    int32_t tok[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) tok[u] = i + u * kThreads < n_hist ? hist[i + u * kThreads] : -1;
#pragma unroll 1
    for (int u = 0; u < 4 && i + u * kThreads < n_hist; ++u)
      count(i + u * kThreads, u == 0 ? tok[0] : (u == 1 ? tok[1] : (u == 2 ? tok[2] : tok[3])));
  }
  if (draft)
    for (int64_t k = tid; k < end - first - 1; k += kThreads) {
      const int32_t tok = draft[k];
      if (tok < 0 || tok >= a.V)
        set_status(a.dev_status, DSPARK_ERR_TOKEN_RANGE);
      else if (tok >= v0 && tok < v0 + width)
        mark((int)(tok - v0));
    }
  for (int64_t k = tid; k < a.bias_cap; k += kThreads) {
    const int32_t *tok = a.bias_tok + r * a.bias_cap;
    if (tok[k] < v0 || tok[k] >= v0 + width) continue;   // -1 pads the list
    bool again = false;
    for (int64_t b = 0; b < k; ++b) again |= tok[b] == tok[k];
    if (again) continue;
    float sum = 0.0f;                                    // a token listed twice: its biases add up in their order
    for (int64_t b = k; b < a.bias_cap; ++b)
      if (tok[b] == tok[k]) sum += a.bias_val[r * a.bias_cap + b];
    biases[atomicAdd(&n_bias, 1)] = Bias{(int32_t)(tok[k] - v0), sum};
    mark((int)(tok[k] - v0));
  }

  // First pass.  Pieces lie on 16-byte boundaries of memory: piece c of a row whose slice starts
  // `shift` elements past one holds elements c N - shift .. + N - 1; those at the ends go element by
  // element.  Where input and output lie differently, all do.
  const T minus_inf = Elem<DT>::from(-INFINITY);
  const T *in0 = reinterpret_cast<const T *>(a.logits) + first * a.V + v0;
  T *out0 = reinterpret_cast<T *>(a.out) + first * a.V + v0;
  const bool in_place = a.logits == a.out;
  const bool alike = (((uintptr_t)a.logits ^ (uintptr_t)a.out) & 15u) == 0;
  const uint32_t pieces = (uint32_t)(width + N - 2) / N + 1;
  const uint32_t items = MASK || !in_place ? (uint32_t)(end - first) * pieces : 0;
  for (uint32_t item0 = tid; item0 < items; item0 += kUnroll * kThreads) {
    uint4 raw[kUnroll];
    int from[kUnroll];
    uint32_t row[kUnroll], bar[kUnroll];
    bool whole[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t item = item0 + u * kThreads;
      row[u] = item / pieces;
      const int shift = (int)(((uintptr_t)(in0 + row[u] * a.V) & 15u) / sizeof(T));
      from[u] = (int)(item - row[u] * pieces) * N - shift;
      whole[u] = item < items && alike && from[u] >= 0 && from[u] + N <= width;
      bar[u] = 0;
      if (MASK && whole[u]) {
        const int64_t v = v0 + from[u], w = v >> 5;
        const int off = (int)(v & 31);
        const uint32_t *mask = a.mask + (first + row[u]) * a.mask_words + w;
        const uint32_t lo = __ldg(mask), hi = off + N > 32 ? __ldg(mask + 1) : 0u;
        bar[u] = ~__funnelshift_r(lo, hi, off) & kAll;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)      // what the mask empties is not read
      if (whole[u] && (!MASK || (bar[u] != kAll && !(in_place && bar[u] == 0))))
        raw[u] = __ldcs(reinterpret_cast<const uint4 *>(in0 + row[u] * a.V + from[u]));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!whole[u]) continue;
      if (MASK) {
        if (in_place && bar[u] == 0) continue;
        uint32_t *x = reinterpret_cast<uint32_t *>(&raw[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (N == 8) {
            const uint32_t lo = (bar[u] >> (2 * i)) & 1 ? 0xff80u : x[i] & 0xffffu;
            x[i] = (bar[u] >> (2 * i + 1)) & 1 ? 0xff800000u | lo : (x[i] & 0xffff0000u) | lo;
          } else {
            x[i] = (bar[u] >> i) & 1 ? 0xff800000u : x[i];
          }
        }
      }
      *reinterpret_cast<uint4 *>(out0 + row[u] * a.V + from[u]) = raw[u];
    }
#pragma unroll 1
    for (int u = 0; u < kUnroll; ++u) {    // the ends
      const uint32_t item = item0 + u * kThreads, j = item / pieces;
      if (item >= items) break;
      const T *in = in0 + j * a.V;
      const int at = (int)(item - j * pieces) * N - (int)(((uintptr_t)in & 15u) / sizeof(T));
      if (alike && at >= 0 && at + N <= width) continue;
      for (int e = max(at, 0); e < min(at + N, width); ++e) {
        const bool allowed = !MASK || ((a.mask[(first + j) * a.mask_words + ((v0 + e) >> 5)] >> ((v0 + e) & 31)) & 1);
        out0[j * a.V + e] = allowed ? in[e] : minus_inf;
      }
    }
  }
  __syncthreads();

  // second pass: the listed tokens
  const int n = n_list;
  const int64_t changes = (int64_t)n * (end - first);
  for (int64_t item = tid; item < changes; item += kThreads) {
    const int j = (int)(item / n), at = list[item - (int64_t)j * n];
    if (MASK && !((a.mask[(first + j) * a.mask_words + ((v0 + at) >> 5)] >> ((v0 + at) & 31)) & 1)) continue;
    T *p = out0 + j * a.V + at;
    float z = Elem<DT>::to(*p);
    uint32_t times = counts[at];
    const bool told = times & kInPrompt;
    times &= ~kInPrompt;
    if (draft)
      for (int k = 0; k < j; ++k) times += draft[k] == (int32_t)(v0 + at);
    if (times || told) z = z > 0.0f ? __fdiv_rn(z, rep) : z * rep;
    if (times) z = z - pre - fre * (float)times;
    for (int b = 0; b < n_bias; ++b)
      if (biases[b].at == at) z += biases[b].sum;
    *p = Elem<DT>::from(z);
  }
}

template <int DT, bool MASK>
cudaError_t launch(const PenalizeArgs &a, cudaStream_t s, int sms) {
  // Larger slices read the history less often, smaller ones give a few requests more CTAs.
  int slice = 8192;
  while (slice > 1024 && a.B * ((a.V + slice - 1) / slice) < 4 * sms) slice /= 2;
  const int64_t bias_slots = a.bias_cap < slice ? a.bias_cap : slice;
  const int smem = slice * 4 + slice / 8 + (int)bias_slots * 8 + slice * 2;
  cudaError_t e = ensure_dynamic_smem((const void *)penalize_kernel<DT, MASK>, smem);
  if (e != cudaSuccess) return e;
  penalize_kernel<DT, MASK><<<(unsigned)(a.B * ((a.V + slice - 1) / slice)), kThreads, smem, s>>>(a, slice);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_penalize(const PenalizeArgs &a, cudaStream_t s, int sms) {
  if (a.dtype == DSPARK_BF16)
    return a.mask ? launch<DSPARK_BF16, true>(a, s, sms) : launch<DSPARK_BF16, false>(a, s, sms);
  return a.mask ? launch<DSPARK_F32, true>(a, s, sms) : launch<DSPARK_F32, false>(a, s, sms);
}

}  // namespace dspark
