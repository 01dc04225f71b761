// xlpk_token_logprobs: log probability, rank, entropy and top alternatives of
// given tokens under rows of logits (include/xlpk.h has the definition).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/xlpk.h"
#include "errors.h"

using namespace xlpk;

namespace {

constexpr int kMaxTop = 64;
constexpr int kThreads = 512;

// A logit's place in descending order: larger keys come first, NaN before +inf,
// -0 equals +0; ties go to the lower index.
__device__ inline uint32_t order_key(float x) {
  if (x != x) return 0xfffffffeu;   // (its bits without the sign are a NaN's again)
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ inline unsigned long long place(float x, int i) {
  return static_cast<unsigned long long>(order_key(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}

// Softmax statistics of a set of logits: the maximum m, and of all others (the
// maximum itself counts 1 and 0, exactly) s = sum e^(x-m), t = sum e^(x-m) (x-m).
struct Stat {
  float m, s, t;
};
__device__ inline Stat join(Stat a, Stat b) {
  if (b.m > a.m) {
    const Stat c = a;
    a = b;
    b = c;
  }
  if (b.m == -INFINITY) return a;
  const float d = b.m - a.m, w = expf(d);   // the smaller side's terms, its maximum among them, move by d
  if (w > 0) {
    a.s += w * (1.f + b.s);
    a.t += w * (b.t + d * (1.f + b.s));
  }
  return a;
}

template <class T>
__device__ inline float logit(const T* x, int i) {
  return static_cast<float>(x[i]);
}

template <class T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const T* logits, int vocab, long long stride, const int* tokens,
                                                            int top_k, float* logprob, float* entropy, int* rank,
                                                            int* top_ids, float* top_logprobs) {
  __shared__ Stat stats[kThreads / 32];
  __shared__ unsigned long long best[kThreads / 32];
  __shared__ int counts[kThreads / 32], nan_seen;
  const long long r = blockIdx.x;
  const T* x = logits + r * stride;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tok = tokens[r];
  const bool valid = tok >= 0 && tok < vocab;
  const float mine = valid ? logit(x, tok) : 0.f;
  const unsigned long long my_place = valid ? place(mine, tok) : 0;
  if (threadIdx.x == 0) nan_seen = 0;
  __syncthreads();
  Stat a{-INFINITY, 0.f, 0.f};
  int before = 0;
  for (int i = threadIdx.x; i < vocab; i += kThreads) {
    const float v = logit(x, i);
    before += place(v, i) > my_place;
    if (v != v || v == INFINITY) nan_seen = 1;
    else a = join(a, Stat{v, 0.f, 0.f});
  }
  for (int o = 16; o; o >>= 1) {
    Stat b{__shfl_xor_sync(~0u, a.m, o), __shfl_xor_sync(~0u, a.s, o), __shfl_xor_sync(~0u, a.t, o)};
    a = join(a, b);
    before += __shfl_xor_sync(~0u, before, o);
  }
  if (lane == 0) stats[warp] = a, counts[warp] = before;
  __syncthreads();
  a = stats[0];
  before = counts[0];
  for (int w = 1; w < kThreads / 32; ++w) a = join(a, stats[w]), before += counts[w];
  const float nan = __int_as_float(0x7fffffff), log_s = log1pf(a.s);
  const bool undefined = nan_seen;
  if (threadIdx.x == 0) {
    logprob[r] = undefined || !valid ? nan : a.m == -INFINITY ? -INFINITY : (mine - a.m) - log_s;
    if (entropy) entropy[r] = undefined ? nan : a.m == -INFINITY ? 0.f : log_s - a.t / (1.f + a.s);
    if (rank) rank[r] = valid ? before : -1;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < top_k; ++k) {
    unsigned long long b = 0;
    for (int i = threadIdx.x; i < vocab; i += kThreads) {
      const unsigned long long c = place(logit(x, i), i);
      if (c < last && c > b) b = c;
    }
    for (int o = 16; o; o >>= 1) {
      const unsigned long long c = __shfl_xor_sync(~0u, b, o);
      if (c > b) b = c;
    }
    __syncthreads();
    if (lane == 0) best[warp] = b;
    __syncthreads();
    b = best[0];
    for (int w = 1; w < kThreads / 32; ++w) b = best[w] > b ? best[w] : b;
    last = b;
    if (threadIdx.x == 0) {
      const float v = key_value(static_cast<uint32_t>(b >> 32));
      top_ids[r * top_k + k] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(b));
      top_logprobs[r * top_k + k] = undefined ? nan : a.m == -INFINITY ? -INFINITY : (v - a.m) - log_s;
    }
  }
}

}  // namespace

extern "C" xlpk_status xlpk_token_logprobs(const void* logits_dev, int32_t dtype, int64_t rows, int32_t vocab,
                                           int64_t row_stride, const int32_t* tokens_dev, int32_t top_k,
                                           float* logprob_dev, float* entropy_dev, int32_t* rank_dev,
                                           int32_t* top_ids_dev, float* top_logprobs_dev, void* stream) {
  if (dtype != XLPK_DTYPE_FP32 && dtype != XLPK_DTYPE_BF16)
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_token_logprobs: dtype is fp32 or bf16");
  if (rows < 0 || vocab < 1 || row_stride < 0 || top_k < 0 || top_k > vocab)
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_token_logprobs: rows, vocab, row_stride or top_k");
  if (top_k > kMaxTop) return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_token_logprobs: top_k over 64");
  if (rows > INT32_MAX) return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_token_logprobs: 2^31 rows or more");
  int sms = 0;
  if (rows > 0) {
    if (!logits_dev || !tokens_dev || !logprob_dev || (top_k > 0 && (!top_ids_dev || !top_logprobs_dev)))
      return refuse(XLPK_ERR_INVALID_ARG, "xlpk_token_logprobs: a pointer is missing");
    if (!aligned(logits_dev, dtype == XLPK_DTYPE_FP32 ? 4 : 2) || !aligned(tokens_dev, 4) || !aligned(logprob_dev, 4) ||
        !aligned(entropy_dev, 4) || !aligned(rank_dev, 4) || !aligned(top_ids_dev, 4) || !aligned(top_logprobs_dev, 4))
      return refuse(XLPK_ERR_INVALID_ARG, "xlpk_token_logprobs: a pointer is not aligned");
  }
  const xlpk_status dev = current_sms(&sms);
  if (dev != XLPK_OK || rows == 0) return dev;
  const dim3 grid(static_cast<unsigned>(rows));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == XLPK_DTYPE_FP32)
    logprobs_kernel<<<grid, kThreads, 0, st>>>(static_cast<const float*>(logits_dev), vocab, row_stride, tokens_dev, top_k,
                                               logprob_dev, entropy_dev, rank_dev, top_ids_dev, top_logprobs_dev);
  else
    logprobs_kernel<<<grid, kThreads, 0, st>>>(static_cast<const __nv_bfloat16*>(logits_dev), vocab, row_stride, tokens_dev,
                                               top_k, logprob_dev, entropy_dev, rank_dev, top_ids_dev, top_logprobs_dev);
  XLPK_CUDA(cudaGetLastError());
  return XLPK_OK;
}
