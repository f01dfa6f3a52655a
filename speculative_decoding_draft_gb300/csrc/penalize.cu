// Penalties for repeated tokens, biases and grammar masks on the logits of ragged rows.
//
// Row i = row_off[r] + j of request r, token v, with n = how often v is among the request's output
// (history from prompt_len on) and the j draft tokens before the row, s = v is in the prompt:
//   z = logit;  if (n > 0 or s) z = z > 0 ? z / repetition : z * repetition
//   z -= presence [n > 0] + frequency n;  z += the request's biases of v;  -inf where the mask bit is 0
// in fp32, rounded once to the logits' type.
//
// One CTA takes one slice of the vocabulary for one request and all of its rows.  It counts the
// history's tokens of its slice once, in shared memory with integer atomics (their order changes
// nothing), streams the rows' slices through and adds a row's draft token to the counts before the
// next row: the history is read once a slice and not once a row.
#include "attn.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kSlice = 4096;                  // tokens of a slice: 16 KB of counts
constexpr uint32_t kInPrompt = 0x80000000u;   // the count's top bit

template <int DT>
__global__ void __launch_bounds__(kThreads) penalize_kernel(const __grid_constant__ PenalizeArgs a) {
  using T = typename Elem<DT>::T;
  extern __shared__ uint32_t counts[];        // [kSlice], then with biases float [kSlice]
  float *bias = reinterpret_cast<float *>(counts + kSlice);
  if (read_status(a.dev_status)) return;
  const int tid = threadIdx.x;
  const int64_t slices = (a.V + kSlice - 1) / kSlice;
  const int64_t r = blockIdx.x / slices, v0 = (blockIdx.x - r * slices) * kSlice;
  const int width = (int)(a.V - v0 < kSlice ? a.V - v0 : kSlice);
  const int64_t first = a.row_off[r], end = a.row_off[r + 1];
  if (first < 0 || end < first || end > a.rows || (a.draft_tok && end - first > a.draft_cap + 1)) {
    if (tid == 0) set_status(a.dev_status, DSPARK_ERR_OFFSETS);
    return;
  }
  const int64_t n_hist = a.hist_len[r], n_prompt = a.prompt_len[r];
  if (n_hist < 0 || n_hist > a.hist_cap || n_prompt < 0 || n_prompt > n_hist) {
    if (tid == 0) set_status(a.dev_status, DSPARK_ERR_LENGTHS);
    return;
  }
  for (int i = tid; i < kSlice; i += kThreads) {
    counts[i] = 0;
    if (a.bias_cap) bias[i] = 0.0f;
  }
  __syncthreads();
  const int32_t *hist = a.hist + r * a.hist_cap;
  for (int64_t i = tid; i < n_hist; i += kThreads) {
    const int32_t tok = hist[i];
    if (tok < 0 || tok >= a.V) {
      set_status(a.dev_status, DSPARK_ERR_TOKEN_RANGE);
    } else if (tok >= v0 && tok < v0 + width) {
      if (i < n_prompt)
        atomicOr(&counts[tok - v0], kInPrompt);
      else
        atomicAdd(&counts[tok - v0], 1u);
    }
  }
  for (int64_t i = tid; i < a.bias_cap; i += kThreads) {
    const int32_t *tok = a.bias_tok + r * a.bias_cap;
    if (tok[i] < v0 || tok[i] >= v0 + width) continue;   // -1 pads the list
    bool again = false;
    for (int64_t k = 0; k < i; ++k) again |= tok[k] == tok[i];
    if (again) continue;
    float sum = 0.0f;                                    // a token listed twice: its biases add up in their order
    for (int64_t k = i; k < a.bias_cap; ++k)
      if (tok[k] == tok[i]) sum += a.bias_val[r * a.bias_cap + k];
    bias[tok[i] - v0] = sum;
  }
  __syncthreads();
  const float rep = a.repetition[r], pre = a.presence[r], fre = a.frequency[r];
  for (int64_t row = first; row < end; ++row) {
    const T *in = reinterpret_cast<const T *>(a.logits) + row * a.V + v0;
    T *out = reinterpret_cast<T *>(a.out) + row * a.V + v0;
    for (int i = tid; i < width; i += kThreads) {
      float z = Elem<DT>::to(in[i]);
      const uint32_t c = counts[i];
      if (c) {
        z = z > 0.0f ? __fdiv_rn(z, rep) : z * rep;
        const uint32_t n = c & ~kInPrompt;
        if (n) z = z - pre - fre * (float)n;
      }
      if (a.bias_cap) z += bias[i];
      if (a.mask && !((a.mask[row * a.mask_words + ((v0 + i) >> 5)] >> ((v0 + i) & 31)) & 1)) z = -INFINITY;
      out[i] = Elem<DT>::from(z);
    }
    if (a.draft_tok && row + 1 < end) {
      __syncthreads();
      if (tid == 0) {
        const int32_t tok = a.draft_tok[r * a.draft_cap + (row - first)];
        if (tok < 0 || tok >= a.V)
          set_status(a.dev_status, DSPARK_ERR_TOKEN_RANGE);
        else if (tok >= v0 && tok < v0 + width)
          counts[tok - v0]++;
      }
      __syncthreads();
    }
  }
}

template <int DT>
cudaError_t launch(const PenalizeArgs &a, cudaStream_t s) {
  const size_t smem = kSlice * (a.bias_cap ? 8 : 4);
  penalize_kernel<DT><<<(unsigned)(a.B * ((a.V + kSlice - 1) / kSlice)), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_penalize(const PenalizeArgs &a, cudaStream_t s) {
  return a.dtype == DSPARK_BF16 ? launch<DSPARK_BF16>(a, s) : launch<DSPARK_F32>(a, s);
}

}  // namespace dspark
