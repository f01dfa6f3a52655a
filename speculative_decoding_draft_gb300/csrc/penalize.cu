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
// large and divergent: 260 us for 288 rows of 151936 where this takes 54.)  In place and without
// a mask the first pass has nothing to do.
#include "attn.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kSlice = 4096;                  // most tokens of a slice
constexpr int kRowsAhead = 2;                 // rows whose loads are in flight together
constexpr int64_t kMaxRequestRows = (1 << 20) - 1;
constexpr uint32_t kInPrompt = 0x80000000u;   // a count's top bit

struct Bias {      // an entry of the request's list that falls into the slice
  int32_t at;
  float value;
  int32_t index;   // in the list
};

template <int DT, bool MASK>
__global__ void __launch_bounds__(kThreads, DT == DSPARK_F32 ? 4 : 5) penalize_kernel(const __grid_constant__ PenalizeArgs a, int slice) {
  using T = typename Elem<DT>::T;
  constexpr int N = 16 / sizeof(T);           // elements of a piece
  constexpr uint32_t kAll = (1u << N) - 1;
  extern __shared__ __align__(16) uint32_t counts[];        // [slice], cleared 16 bytes at a time
  uint32_t *map = counts + slice;             // [slice / 32]: listed tokens
  Bias *biases = reinterpret_cast<Bias *>(map + slice / 32);                        // [bias_cap], in no order
  uint16_t *list = reinterpret_cast<uint16_t *>(biases + a.bias_cap);               // [slice]
  __shared__ int n_list, n_bias;
  const int tid = threadIdx.x;
  const int slices = (int)((a.V + slice - 1) / slice);
  const int r = (int)(blockIdx.x / (unsigned)slices), V = (int)a.V;      // V <= 2^30, B <= 2^20
  const int v0 = (int)(blockIdx.x - (unsigned)(r * slices)) * slice, width = min(V - v0, slice);
  const int status = status_on_entry(a.dev_status);
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
  const int32_t *hist = a.hist + (int64_t)r * a.hist_cap;
  const int32_t *draft = a.draft_tok ? a.draft_tok + (int64_t)r * a.draft_cap : nullptr;
  auto mark = [&](int at) {
    const uint32_t bit = 1u << (at & 31);
    if (!(atomicOr(&map[at >> 5], bit) & bit)) list[atomicAdd(&n_list, 1)] = (uint16_t)at;
  };
  const int told = (int)n_prompt, heard = (int)n_hist;
  auto count = [&](int i, int32_t tok) {
    const uint32_t at = (uint32_t)(tok - v0);
    if (at < (uint32_t)width) {                          // a token of the slice, and so of the vocabulary
      if (i < told)
        atomicOr(&counts[at], kInPrompt);
      else
        atomicAdd(&counts[at], 1u);
      mark((int)at);
    } else if ((uint32_t)tok >= (uint32_t)V) {
      set_status(a.dev_status, DSPARK_ERR_TOKEN_RANGE);
    }
  };
  for (int i = tid; i < heard; i += 4 * kThreads) {
    int32_t tok[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) tok[u] = i < heard - u * kThreads ? hist[i + u * kThreads] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i < heard - u * kThreads) count(i + u * kThreads, tok[u]);
  }
  if (draft)
    for (int64_t k = tid; k < end - first - 1; k += kThreads) {
      const int32_t tok = draft[k];
      if (tok < 0 || tok >= V)
        set_status(a.dev_status, DSPARK_ERR_TOKEN_RANGE);
      else if (tok >= v0 && tok < v0 + width)
        mark((int)(tok - v0));
    }
  for (int k = tid; k < (int)a.bias_cap; k += kThreads) {
    const uint32_t at = (uint32_t)(a.bias_tok[(int64_t)r * a.bias_cap + k] - v0);
    if (at >= (uint32_t)width) continue;                 // another slice's, or the padding's -1
    biases[atomicAdd(&n_bias, 1)] = Bias{(int32_t)at, a.bias_val[(int64_t)r * a.bias_cap + k], k};
    mark((int)at);
  }

  // First pass.  Pieces lie on 16-byte boundaries of memory; what a row's slice has before its first
  // boundary and after its last goes element by element, and so does all of it where input and output
  // lie differently.
  const T minus_inf = Elem<DT>::from(-INFINITY);
  const T *in0 = reinterpret_cast<const T *>(a.logits) + first * a.V + v0;
  T *out0 = reinterpret_cast<T *>(a.out) + first * a.V + v0;
  const bool in_place = a.logits == a.out;
  const bool alike = (((uintptr_t)a.logits ^ (uintptr_t)a.out) & 15u) == 0;
  constexpr int kPer = kSlice / N / kThreads;       // pieces of a row's slice for a thread
  const int n_rows = MASK || !in_place ? (int)(end - first) : 0;
  const int64_t over = reinterpret_cast<char *>(out0) - reinterpret_cast<const char *>(in0);   // from input to output
  const T *in = in0;
  const uint32_t *mask = MASK ? a.mask + first * a.mask_words + (v0 >> 5) : nullptr;   // slices begin at words
  for (int j0 = 0; j0 < n_rows; j0 += kRowsAhead) {
    uint4 raw[kRowsAhead][kPer];
    uint32_t bar[kRowsAhead][kPer];                  // tokens that the mask forbids; ~0: no piece
    const uint4 *body[kRowsAhead];
#pragma unroll
    for (int r = 0; r < kRowsAhead; ++r) {
      const int before = (int)((0u - (uint32_t)(uintptr_t)in) & 15u) / (int)sizeof(T);
      const int head = alike && before < width ? before : width, pieces = j0 + r < n_rows ? (width - head) / N : 0;
      body[r] = reinterpret_cast<const uint4 *>(in + head) + tid;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int p = tid + k * kThreads;
        bar[r][k] = ~0u;
        if (p < pieces) {
          bar[r][k] = 0;
          if (MASK) {
            const int at = head + p * N, off = at & 31;
            const uint32_t *m = mask + (at >> 5);
            bar[r][k] = ~__funnelshift_r(__ldg(m), off + N > 32 ? __ldg(m + 1) : 0u, off) & kAll;
          }
        }
      }
      in += a.V;
      if (MASK) mask += a.mask_words;
    }
#pragma unroll
    for (int r = 0; r < kRowsAhead; ++r)             // what the mask empties is not read
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (bar[r][k] != ~0u && (!MASK || (bar[r][k] != kAll && !(in_place && bar[r][k] == 0))))
          raw[r][k] = __ldcs(body[r] + k * kThreads);
#pragma unroll
    for (int r = 0; r < kRowsAhead; ++r) {
      uint4 *to = reinterpret_cast<uint4 *>(reinterpret_cast<uintptr_t>(body[r]) + over);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const uint32_t b = bar[r][k];
        if (b == ~0u || (MASK && in_place && b == 0)) continue;
        if (MASK && b) {
          uint32_t *x = reinterpret_cast<uint32_t *>(&raw[r][k]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (N == 8) {
              // the bits of a word's two halves, moved to the top of a byte and spread over two each
              uint32_t m;
              asm("prmt.b32 %0, %1, %2, 0xCC88;" : "=r"(m) : "r"((b << 7) >> (2 * i)), "r"((b << 6) >> (2 * i)));
              x[i] = (x[i] & ~m) | (0xff80ff80u & m);
            } else {
              x[i] = (b >> i) & 1 ? 0xff800000u : x[i];
            }
          }
        }
        to[k * kThreads] = raw[r][k];
      }
    }
  }
  for (int j = tid / 32; j < n_rows; j += kThreads / 32) {      // the rows' ends, a warp a row
    const T *in = in0 + j * a.V;
    const int before = (int)((0u - (uint32_t)(uintptr_t)in) & 15u) / (int)sizeof(T);
    const int head = alike && before < width ? before : width, tail = head + (width - head) / N * N;
    for (int e = tid % 32; e < head + width - tail; e += 32) {
      const int at = e < head ? e : tail + e - head;
      const bool allowed = !MASK || ((a.mask[(first + j) * a.mask_words + ((v0 + at) >> 5)] >> (at & 31)) & 1);
      out0[j * a.V + at] = allowed ? in[at] : minus_inf;
    }
  }
  __syncthreads();

  // second pass: the listed tokens
  const int n = n_list;
  const uint32_t changes = (uint32_t)n * (uint32_t)(end - first);       // up to 2^12 * 2^20
  for (uint32_t item = tid; item < changes; item += kThreads) {
    const int j = (int)(item / (uint32_t)n), at = list[item - (uint32_t)(j * n)];
    if (MASK && !((a.mask[(first + j) * a.mask_words + ((v0 + at) >> 5)] >> ((v0 + at) & 31)) & 1)) continue;
    T *p = out0 + j * a.V + at;
    float z = Elem<DT>::to(*p);
    uint32_t times = counts[at];
    const bool prompted = times & kInPrompt;
    times &= ~kInPrompt;
    if (draft)
      for (int k = 0; k < j; ++k) times += draft[k] == (int32_t)(v0 + at);
    if (times || prompted) z = z > 0.0f ? __fdiv_rn(z, rep) : z * rep;
    if (times) z = z - pre - fre * (float)times;
    float sum = 0.0f;                                    // a token listed twice: its biases add up in the list's order
    for (int done = -1, next = 0; n_bias > 0 && next < INT32_MAX; done = next) {
      float value = 0.0f;
      next = INT32_MAX;
      for (int b = 0; b < n_bias; ++b)
        if (biases[b].at == at && biases[b].index > done && biases[b].index < next) next = biases[b].index, value = biases[b].value;
      sum += value;
    }
    z += sum;
    *p = Elem<DT>::from(z);
  }
}

template <int DT, bool MASK>
cudaError_t launch(const PenalizeArgs &a, cudaStream_t s, int sms) {
  // Larger slices read the history less often, smaller ones give a few requests more CTAs.
  int slice = kSlice;
  while (slice > 1024 && a.B * ((a.V + slice - 1) / slice) < 4 * sms) slice /= 2;
  const int smem = slice * 4 + slice / 8 + (int)a.bias_cap * (int)sizeof(Bias) + slice * 2;
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
