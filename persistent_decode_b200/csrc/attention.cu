// xlpk_decode_attention: attention of one new token per sequence over its KV
// cache (include/xlpk.h has the definition).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/xlpk.h"
#include "errors.h"

using namespace xlpk;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ inline float load_io(const void* p, long long i, int io) {
  return io == XLPK_DTYPE_FP32 ? static_cast<const float*>(p)[i]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ inline void store_io(void* p, long long i, int io, float v) {
  if (io == XLPK_DTYPE_FP32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
__device__ inline float load_kv(const void* p, long long i, int kv, float scale) {
  if (kv == XLPK_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  __nv_fp8_e4m3 c;
  c.__x = static_cast<const uint8_t*>(p)[i];
  return static_cast<float>(c) * scale;
}
// Stores x as a cache entry and returns the value the entry stands for.
__device__ inline float round_kv(void* p, long long i, int kv, float scale, float x, bool store) {
  if (kv == XLPK_DTYPE_BF16) {
    const __nv_bfloat16 b = __float2bfloat16_rn(x);
    if (store) static_cast<__nv_bfloat16*>(p)[i] = b;
    return __bfloat162float(b);
  }
  __nv_fp8_e4m3 c(x / scale);
  if (store) static_cast<uint8_t*>(p)[i] = c.__x;
  return static_cast<float>(c) * scale;
}

// One block per (sequence, query head), its warps stepping through the visible
// positions with an online softmax each, merged at the end.
constexpr int kWarps = 4;

__global__ void attention_kernel(const xlpk_attention_args a) {
  const int h = blockIdx.x, b = blockIdx.y, g = a.n_q_heads / a.n_kv_heads, kh = h / g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = a.head_dim / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][128];
  __shared__ int bad_page;
  if (threadIdx.x == 0) bad_page = 0;
  __syncthreads();
  const long long cap = static_cast<long long>(a.table_cols) * a.page_size;
  int n = a.seq_lens_dev[b];
  bool bad = n < 0 || n > cap;
  if (bad) n = 0;
  const int lo = a.window > 0 && n > a.window ? n - a.window : 0;
  const int first = a.sinks < lo ? a.sinks : lo;   // [0, first) and [lo, n)
  const int count = first + (n - lo);
  float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0;
  for (int i = 0; i < per; ++i)
    q[i] = load_io(a.q_dev, b * a.q_seq_stride + h * a.q_head_stride + lane + 32 * i, a.io_dtype);
  const float s2 = a.scale * kLog2e;
  for (int v = warp; v < count; v += kWarps) {
    const int t = v < first ? v : lo + (v - first);
    const int j = t / a.page_size, r = t - j * a.page_size;
    const long long page = a.page_table_dev ? a.page_table_dev[b * a.table_stride + j] : b;
    if (page < 0 || page >= a.n_pages) {
      bad_page = 1;
      continue;
    }
    const long long ko = page * a.k_page_stride + kh * a.k_head_stride + r * a.k_pos_stride;
    const long long vo = page * a.v_page_stride + kh * a.v_head_stride + r * a.v_pos_stride;
    const bool fresh = a.k_new_dev && t == n - 1;
    float s = 0, vv[4];
    for (int i = 0; i < per; ++i) {
      const int e = lane + 32 * i;
      float k;
      if (fresh) {
        k = round_kv(a.k_dev, ko + e, a.kv_dtype, a.k_scale,
                     load_io(a.k_new_dev, b * a.new_k_seq_stride + kh * a.new_k_head_stride + e, a.io_dtype), h == kh * g);
        vv[i] = round_kv(a.v_dev, vo + e, a.kv_dtype, a.v_scale,
                         load_io(a.v_new_dev, b * a.new_v_seq_stride + kh * a.new_v_head_stride + e, a.io_dtype), h == kh * g);
      } else {
        k = load_kv(a.k_dev, ko + e, a.kv_dtype, a.k_scale);
        vv[i] = load_kv(a.v_dev, vo + e, a.kv_dtype, a.v_scale);
      }
      s += q[i] * k;
    }
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    s *= s2;
    const float mn = s > m || s != s ? s : m;   // NaN stays
    const float w = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(s - mn);
    l = l * w + p;
    for (int i = 0; i < per; ++i) o[i] = o[i] * w + p * vv[i];
    m = mn;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int i = 0; i < per; ++i) so[warp][lane + 32 * i] = o[i];
  __syncthreads();
  if (threadIdx.x >= a.head_dim) return;
  float M = -INFINITY, L = 0, O = 0;
  for (int w = 0; w < kWarps; ++w) M = sm[w] > M || sm[w] != sm[w] ? sm[w] : M;
  for (int w = 0; w < kWarps; ++w) {
    const float f = M == -INFINITY ? 0.f : exp2f(sm[w] - M);
    L += sl[w] * f;
    O += so[w][threadIdx.x] * f;
  }
  bad = bad || bad_page;
  const float nan = __int_as_float(0x7fffffff);
  const float out = bad ? nan : L == 0 ? 0.f : O / L;
  store_io(a.out_dev, b * a.out_seq_stride + h * a.out_head_stride + threadIdx.x, a.io_dtype, out);
  if (threadIdx.x == 0) {
    if (a.lse_dev)
      a.lse_dev[static_cast<long long>(b) * a.n_q_heads + h] = bad ? nan : L == 0 ? -INFINITY : M * kLn2 + logf(L);
    if (bad && a.status_dev) *a.status_dev = XLPK_ERR_INVALID_ARG;
  }
}

bool power_of_two_scale(float s) {
  if (!(s >= 0x1p-24f && s <= 0x1p24f)) return false;
  int e;
  return std::frexp(s, &e) == 0.5f;
}

bool shape_ok(const xlpk_attention_args* a) {
  return a && a->n_seqs >= 0 && a->n_q_heads > 0 && a->n_kv_heads > 0 && a->n_q_heads % a->n_kv_heads == 0 &&
         a->head_dim > 0;
}

xlpk_status check_args(const xlpk_attention_args* a) {
  if (!a) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: no arguments");
  if (!shape_ok(a)) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: n_seqs, heads or head_dim");
  if ((a->head_dim != 64 && a->head_dim != 128) || a->n_q_heads / a->n_kv_heads > 16)
    return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_decode_attention: head_dim 64 or 128, at most 16 query heads per kv head");
  if ((a->io_dtype != XLPK_DTYPE_BF16 && a->io_dtype != XLPK_DTYPE_FP32) ||
      (a->kv_dtype != XLPK_DTYPE_BF16 && a->kv_dtype != XLPK_DTYPE_FP8_E4M3))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: io_dtype is bf16 or fp32, kv_dtype bf16 or e4m3");
  if (a->n_pages < 0 || a->page_size < 1 || a->table_cols < 0 || a->window < 0 || a->sinks < 0)
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: a negative count");
  if (static_cast<int64_t>(a->table_cols) * a->page_size > INT32_MAX)
    return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_decode_attention: a table of 2^31 positions or more");
  if (!(a->scale > 0) || !std::isfinite(a->scale))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: scale is not finite and positive");
  if (a->kv_dtype == XLPK_DTYPE_FP8_E4M3 && (!power_of_two_scale(a->k_scale) || !power_of_two_scale(a->v_scale)))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: cache scales are powers of two in [2^-24, 2^24]");
  if (a->n_seqs == 0) return XLPK_OK;
  if (!a->q_dev || !a->seq_lens_dev || !a->out_dev || (!a->k_new_dev) != (!a->v_new_dev) ||
      ((!a->k_dev || !a->v_dev) && a->n_pages > 0))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: a pointer is missing");
  if (!a->page_table_dev && (a->table_cols != 1 || a->n_pages != a->n_seqs))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: a contiguous cache has one page per sequence");
  const int64_t io = a->io_dtype == XLPK_DTYPE_FP32 ? 4 : 2, kv = a->kv_dtype == XLPK_DTYPE_BF16 ? 2 : 1;
  const int64_t io_strides[] = {a->q_seq_stride,      a->q_head_stride,     a->new_k_seq_stride, a->new_k_head_stride,
                                a->new_v_seq_stride,  a->new_v_head_stride, a->out_seq_stride,   a->out_head_stride};
  const int64_t kv_strides[] = {a->k_page_stride, a->k_head_stride, a->k_pos_stride,
                                a->v_page_stride, a->v_head_stride, a->v_pos_stride};
  bool ok = aligned(a->q_dev, 16) && aligned(a->out_dev, 16) && aligned(a->k_new_dev, 16) && aligned(a->v_new_dev, 16) &&
            aligned(a->k_dev, 16) && aligned(a->v_dev, 16) && aligned(a->page_table_dev, 4) &&
            aligned(a->seq_lens_dev, 4) && aligned(a->lse_dev, 4) && aligned(a->status_dev, 4);
  for (int64_t s : io_strides) ok = ok && (s * io) % 16 == 0;
  for (int64_t s : kv_strides) ok = ok && (s * kv) % 16 == 0;
  if (!ok) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: a pointer or stride is not a multiple of 16 bytes");
  return XLPK_OK;
}

}  // namespace

extern "C" int64_t xlpk_decode_attention_workspace(const xlpk_attention_args* a) { return shape_ok(a) ? 16 : 0; }

extern "C" xlpk_status xlpk_decode_attention(const xlpk_attention_args* a, void* workspace_dev, int64_t workspace_bytes,
                                             void* stream) {
  const xlpk_status rc = check_args(a);
  if (rc != XLPK_OK) return rc;
  if (!workspace_dev || !aligned(workspace_dev, 16) || workspace_bytes < xlpk_decode_attention_workspace(a))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: workspace missing, unaligned or too small");
  int sms = 0;
  const xlpk_status dev = current_sms(&sms);
  if (dev != XLPK_OK) return dev;
  if (a->n_seqs == 0) return XLPK_OK;
  if (a->n_seqs > 65535) return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_decode_attention: more than 65535 sequences");
  attention_kernel<<<dim3(a->n_q_heads, a->n_seqs), kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(*a);
  XLPK_CUDA(cudaGetLastError());
  return XLPK_OK;
}
