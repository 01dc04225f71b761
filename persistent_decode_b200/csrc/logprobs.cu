// xlpk_token_logprobs: log probability, rank, entropy and top alternatives of
// given tokens under rows of logits (include/xlpk.h has the definition).
//
// Mathematics.  With m the largest logit, s = sum of e^(x-m) over all others and
// t = sum of e^(x-m) (x-m): logprob = (x_tok - m) - log1p(s), entropy =
// log1p(s) - t / (1 + s).  The maximum itself is kept out of s, so that the log
// probability of a nearly certain token keeps its digits.  Two sets join by
// moving the smaller maximum's sums (join).
//
// One pass: each logit is read once from memory, in 16-byte vectors that the
// thread which uses them copies into its own queue in shared memory.  A row is
// one CTA's, or, with few rows, a cluster's of up to 8 CTAs, joined through
// distributed shared memory: no workspace and one launch.
//
// Alternatives.  The (k+1)-th largest of 64 or 128 groups' maxima bounds the k-th
// largest logit from below, and closely: in random order about k + k/4 logits
// pass it for k = 20, 90 for 64.  They are found again where a thread's marks say
// so, and ranked by counting.
//
// Bound (times of a captured call replayed, on the device; among calls through
// Python they are 2 to 10 us longer): 1024 rows of 128256 fp32 logits take 96 us, 85%
// of the copy rate (109 with 20 alternatives); rows of bf16 by the instructions for
// each logit and the uneven rows of each SM (333 rows of 64007 take 20 us, 29 with 64
// alternatives, of which 6.6 are memory; no pipe is saturated); single rows by latency
// (32000: 4.4 us, 7.2 with 5 alternatives).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/xlpk.h"
#include "errors.h"

using namespace xlpk;

namespace {

constexpr int kMaxTop = 64;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kGroups = 128;       // most groups of threads, each known by its largest logit
constexpr int kMarks = 32;         // stretches of rounds that a thread knows its largest logit of
constexpr int kUnroll = 4;         // 16-byte vectors a thread takes in a round
constexpr int kStages = 2;         // rounds on their way
constexpr int kStep = kUnroll * kThreads;
constexpr int kPushed = 512;       // candidates that are ranked at most
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A maximum this far out has no neighbour within 64, so all others weigh less than 2^-92 and are left
// out.  Nearer ones have a base, m log2(e) rounded, that is off by 64 at most, which exponentials of it
// stand; further out what the rounding leaves is an exponent of its own (-1e10: 440).
constexpr float kFar = 0x1p30f;

// A logit's place in descending order: larger keys come first, NaN before +inf,
// -0 equals +0; ties go to the lower index.  No value has key 0.
__device__ inline uint32_t order_key(float x) {
  if (x != x) return 0xfffffffeu;   // (its bits without the sign are a NaN's again)
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
// The key below k (no value has the key of -0).
__device__ inline uint32_t key_below(uint32_t k) { return k - (k == 0x80000000u ? 2 : 1); }
__device__ inline unsigned long long place(float x, int i) {
  return static_cast<unsigned long long>(order_key(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ inline int place_index(unsigned long long p) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(p)); }

// 2^x to 2^-22, 0 for -inf.
__device__ inline float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The larger; NaN if either is.
__device__ inline float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ inline float warp_max_nan(float x) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ inline float warp_sum(float x) {
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// Softmax statistics of a set of logits: the maximum m, and of all others (the
// maximum itself counts 1 and 0, exactly) s = sum e^(x-m), t = sum e^(x-m) (x-m).
// The others are kept apart so that log(1 + s) keeps a small s.  NaN in t: the
// set holds NaN or +inf.
struct Stat {
  float m, s, t;
};
__device__ inline Stat join(Stat a, Stat b) {
  if (b.m > a.m) {
    const Stat c = a;
    a = b;
    b = c;
  }
  if (b.m == -INFINITY) {
    a.t += b.t;   // 0, or the NaN of a part of nothing but NaN
    return a;
  }
  const float d = b.m - a.m, w = ex2(d * kLog2e);   // b's terms, its maximum among them, move by d
  a.s += w * (1.f + b.s);
  a.t += w > 0.f ? w * (b.t + d * (1.f + b.s)) : w * b.t;
  return a;
}

template <class T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  static constexpr uint32_t NONE = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;   // -inf
  uint4 v;
  __device__ float operator[](int i) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  // How many are not <= `bar` (a value of T), or, with `equal`, not < it.
  __device__ int before(float bar, bool equal) const {
    int n = 0;
    if (sizeof(T) == 4) {
      const float b = !equal ? bar : bar == -INFINITY ? __int_as_float(0x7fffffff) : key_value(key_below(order_key(bar)));
#pragma unroll
      for (int i = 0; i < N; ++i)
        asm("{ .reg .pred p; setp.gtu.f32 p, %1, %2; @p add.s32 %0, %0, 1; }" : "+r"(n) : "f"((*this)[i]), "f"(b));
      return n;
    }
    // two at a time, as 1 and 0, which bf16 adds exactly
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 b = __float2bfloat162_rn(bar);
    __nv_bfloat162 sum = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = __hadd2(sum, equal ? __hgeu2(p[i], b) : __hgtu2(p[i], b));
    return static_cast<int>(__low2float(sum) + __high2float(sum));
  }
  // NaN if there is one
  __device__ float largest() const {
    if (sizeof(T) == 4) return max_nan(max_nan((*this)[0], (*this)[1]), max_nan((*this)[2], (*this)[3]));
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
    return max_nan(__low2float(m), __high2float(m));
  }
};

// What one thread gathers of its part of a row.  Terms are kept as powers of 2: with
// y = x log2(e) - base, rounded once, s = sum 2^y and t = sum 2^y y over the logits below
// the warp's maximum m; base is m log2(e) rounded, and what that leaves, y of m itself, is
// put right at the end.  Against x - m, a product and an exponential this saves an instruction
// for each logit.
struct Gather {
  float m = -INFINITY, base = 0.f, s = 0.f, t = 0.f;
  int ties = 0;            // logits equal to m
  int before = 0;          // logits that come before the token's
  bool careful = false;    // logits of -inf have been met: 2^y y is 0 times infinity

  __device__ float own() const { return fmaf(m, kLog2e, -base); }
  // A logit that may be the maximum; NaN, and +inf, leave NaN in t.
  __device__ void any(float x) {
    if (x < m) {
      const float y = fmaxf(fmaf(x, kLog2e, -base), -1000.f), e = ex2(y);
      s += e;
      t += e * y;
    } else {
      ++ties;
      t += x - m;
    }
  }
  __device__ void rise(float top) {
    const float up = fminf(fmaxf(top * kLog2e, -3e38f), 3e38f);
    if (fabsf(m) < kFar) {
      const float y = own(), e = ties * ex2(y), d = base - up, w = ex2(d);
      t += e * y;
      s += e;
      t = w > 0.f ? w * (t + d * s) : w * t;
      s *= w;
    } else {
      s = 0.f;
      t = t != t ? t : 0.f;
    }
    ties = 0;
    m = top;
    base = up;
  }
};

constexpr int kQueueBytes = kStages * kStep * 16;

struct alignas(16) Shared {
  unsigned long long pushed[kMaxCluster * kMaxTop];
  unsigned long long lists[kMaxCluster][kMaxTop];   // the leader's: every part's top tokens
  __nv_bfloat16 marks[kMarks][kThreads];            // rounded up
  uint32_t groups[kGroups];                         // largest key of each group
  Stat stats[kMaxCluster];
  int befores[kMaxCluster];
  uint32_t bar;                                     // key: at least top_k + 1 groups have a larger one or this
  Stat warp_stats[kWarps];
  int warp_befores[kWarps], warp_counts[kWarps];
  unsigned long long best[kWarps];
  int n_pushed;
};
static_assert(kPushed <= kMaxCluster * kMaxTop, "candidates");

// Statistics and rank of one round: the thread's vectors, those past the part's end all -inf,
// which adds nothing to either (`left`: the vectors wholly to the left of the token that the part
// has; `mine`: the token's logit); `top` the warp's largest logit, or NaN.
template <class T>
__device__ inline void round_stats(Gather& g, const Vec<T> (&v)[kUnroll], float top, int first, int left, float mine) {
  constexpr int N = Vec<T>::N;
  if (!(top < mine)) {   // (few rounds have larger ones if it is a likely token)
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) g.before += v[u].before(mine, first + u * kThreads < left);
  }
  float x[kUnroll * N];
#pragma unroll
  for (int i = 0; i < kUnroll * N; ++i) x[i] = v[i / N][i % N];
  if (top >= g.m) {
    if (top > g.m) g.rise(top);
    if (top == -INFINITY) return;
    // the maximum stands here: it is counted, and what is added in its place is 0
    const float far = top - fmaxf(700.f, fabsf(top));   // (NaN for +inf)
#pragma unroll
    for (int i = 0; i < kUnroll * N; ++i)
      if (x[i] == top) x[i] = far, ++g.ties;
  }
  float s = 0.f, t = 0.f;
  if (!g.careful) {
#pragma unroll
    for (int i = 0; i < kUnroll * N; ++i) {
      const float y = fmaf(x[i], kLog2e, -g.base), e = ex2(y);
      s += e;
      t = fmaf(e, y, t);
    }
    g.careful = t != t;
  }
  if (g.careful) {
    s = t = 0.f;
#pragma unroll
    for (int i = 0; i < kUnroll * N; ++i) {
      const float y = max_nan(fmaf(x[i], kLog2e, -g.base), -1000.f), e = ex2(y);
      s += e;
      t = fmaf(e, y, t);
    }
  }
  g.s += s;
  g.t += t;
}

// Raises the bar to the (top_k + 1)-th largest of the groups' keys: at least so many logits
// are that large, so no smaller one is an alternative.  Threads 0 .. groups - 1 call it.
__device__ inline void raise_bar(Shared& sh, int groups, int top_k) {
  const uint4* keys = reinterpret_cast<const uint4*>(sh.groups);
  const uint32_t mine = sh.groups[threadIdx.x];
  int at_least = 0;
#pragma unroll 8
  for (int i = 0; i < groups / 4; ++i) {
    const uint4 k = keys[i];
    at_least += (k.x >= mine) + (k.y >= mine) + (k.z >= mine) + (k.w >= mine);
  }
  if (at_least > top_k) atomicMax(&sh.bar, mine);
}

__device__ inline void push(Shared& sh, float x, int index) {
  const int at = atomicAdd(&sh.n_pushed, 1);
  if (at < kPushed) sh.pushed[at] = place(x, index);
}

// Ranks a list in shared memory: out[0 .. top_k) gets its largest, the rest of out is left.
__device__ inline void rank_list(const unsigned long long* list, int n, int top_k, unsigned long long* out) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long mine = list[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) r += list[j] > mine;
    if (r < top_k) out[r] = mine;
  }
}

// One cluster per row, its CTAs taking consecutive parts.
template <class T>
__global__ void __launch_bounds__(kThreads, 3) logprobs_kernel(const T* logits, int vocab, long long stride, const int* tokens,
                                                               int top_k, int parts, float* logprob, float* entropy, int* rank,
                                                               int* top_ids, float* top_logprobs) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  constexpr int N = Vec<T>::N;
  const long long r = blockIdx.x / parts;
  const int part = blockIdx.x - static_cast<int>(r) * parts;
  const T* x = logits + r * stride;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed;");   // this CTA runs: its memory may be written
  // whole vectors of the row are [pre, pre + N * vecs); what is left at its ends goes to the first and last part
  const int pre = min(vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
  const int vecs = (vocab - pre) / N, v0 = static_cast<int>(static_cast<long long>(vecs) * part / parts),
            v1 = static_cast<int>(static_cast<long long>(vecs) * (part + 1) / parts);
  const int lo = part == 0 ? 0 : pre + v0 * N, hi = part == parts - 1 ? vocab : pre + v1 * N;
  const uint4* const body = reinterpret_cast<const uint4*>(x + pre);

  // Every thread copies the bytes that it reads itself, so its own wait is the only one.
  Vec<T>* const queue = reinterpret_cast<Vec<T>*>(raw + sizeof(Shared)) + threadIdx.x;
  const uint32_t queue_at = static_cast<uint32_t>(__cvta_generic_to_shared(queue));
  const auto fetch = [&](int from, int stage) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (from + u * kThreads < v1)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(queue_at + (stage * kStep + u * kThreads) * 16),
                     "l"(body + from + u * kThreads)
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int mine0 = v0 + threadIdx.x;   // the thread's first vector
  for (int i = 0; i < kStages; ++i) fetch(mine0 + i * kStep, i);
  const int tok = tokens[r];
  const bool valid = tok >= 0 && tok < vocab;
  const float mine = valid ? static_cast<float>(x[tok]) : 0.f;
  if (threadIdx.x < kGroups) sh.groups[threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.n_pushed = 0, sh.bar = 0;
  __syncthreads();

  // A logit comes before the token's if it is not <= it, or, to the left of the token, not < it.
  // tok_vec: the vectors wholly to the left.
  const int tok_vec = tok < pre ? 0 : (tok - pre) / N, left = min(tok_vec, v1);
  const uint32_t my_key = order_key(mine);

  // the ends, one logit of a thread at most
  Gather g;
  float best = -INFINITY;   // the thread's largest logit, or NaN
  int end_at = -1;
  if (part == 0 && static_cast<int>(threadIdx.x) < pre) end_at = threadIdx.x;
  if (part == parts - 1 && static_cast<int>(threadIdx.x) >= 32 && pre + vecs * N + static_cast<int>(threadIdx.x) - 32 < vocab)
    end_at = pre + vecs * N + threadIdx.x - 32;
  const float end = end_at >= 0 ? static_cast<float>(x[end_at]) : -INFINITY;
  if (warp < 2) {
    const float top = warp_max_nan(end);
    if (top > -INFINITY) g.rise(top);
    if (end_at >= 0) {
      if (top > -INFINITY) g.any(end);
      g.before = !(end <= mine) || (end_at < tok && !(end < mine));
      best = end;
    }
    if (top != top) g.t = top;
  }

  // ---- the row streams by
  const int rounds = (v1 - v0 + kStep - 1) / kStep;
  int shift = 0;
  while (rounds >> shift >= kMarks) ++shift;   // rounds to a mark: 2^shift
  int stage = 0, first = mine0;
#pragma unroll 1
  for (int round = 0; round < rounds; ++round, first += kStep) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    Vec<T> v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = queue[stage * kStep + u * kThreads];
    if (round == rounds - 1) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (first + u * kThreads >= v1) v[u].v = make_uint4(Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE);
    }
    float top = v[0].largest();
#pragma unroll
    for (int u = 1; u < kUnroll; ++u) top = max_nan(top, v[u].largest());
    best = max_nan(best, top);
    if (top_k > 0) {
      __nv_bfloat16* const mark = &sh.marks[round >> shift][threadIdx.x];
      *mark = __float2bfloat16_ru(round & ((1 << shift) - 1) ? max_nan(__bfloat162float(*mark), top) : top);
    }
    top = warp_max_nan(top);
    round_stats<T>(g, v, top, first, left, mine);
    // (a part that fits in the queue stays there)
    if (round + kStages < rounds) fetch(first + kStages * kStep, stage);
    else asm volatile("cp.async.commit_group;" ::: "memory");
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }

  // ---- this part's statistics
  {
    float s = warp_sum(g.s), t = warp_sum(g.t);
    const int ties = __reduce_add_sync(~0u, g.ties), before = __reduce_add_sync(~0u, g.before);
    if (fabsf(g.m) < kFar) {
      const float y = g.own(), f = ex2(-y);
      t = (t - y * s) * f * kLn2;
      s = s * f + (ties - 1);
    } else {
      s = g.m == -INFINITY ? 0.f : static_cast<float>(ties - 1);
      t = t != t ? t : 0.f;
    }
    if (lane == 0) {
      sh.warp_stats[warp] = {g.m, s, t};
      sh.warp_befores[warp] = before;
    }
  }
  const int groups = top_k < kGroups / 4 ? kGroups / 2 : kGroups;   // about twice top_k or more
  if (top_k > 0 && (mine0 < v1 || end_at >= 0)) atomicMax(&sh.groups[threadIdx.x & (groups - 1)], order_key(best));
  __syncthreads();
  Stat all = sh.warp_stats[0];
  int before = 0;
  if (warp == kWarps - 1) {
    // joined in the order of the warps
    for (int w = 1; w < kWarps; ++w) all = join(all, sh.warp_stats[w]);
    before = __reduce_add_sync(~0u, lane < kWarps ? sh.warp_befores[lane] : 0);
    if (valid && mine != mine) {
      // a NaN's rank: the NaN to its left
      before = 0;
      for (int i = lo + lane; i < min(hi, tok); i += 32) before += order_key(static_cast<float>(x[i])) == my_key;
      before = __reduce_add_sync(~0u, before);
    } else if (valid && tok >= pre && tok_vec >= v0 && tok_vec < v1) {
      // equals to the left of the token in its own vector
      const int i = pre + tok_vec * N + lane;
      before += __reduce_add_sync(~0u, static_cast<int>(i < tok && static_cast<float>(x[min(i, tok)]) == mine));
    }
  }

  // ---- this part's top tokens, in order
  const int want = min(top_k, hi - lo);
  unsigned long long* const out = sh.lists[0];
  if (top_k > 0) {
    if (static_cast<int>(threadIdx.x) < groups) raise_bar(sh, groups, top_k);
    __syncthreads();
    // The candidates are the logits that the bar lets through, found again where a thread's mark says
    // that there are some: about as many of its stretches as there are alternatives.  (Listing them
    // while the row streams by, under a bar that rises, took more instructions than the statistics:
    // 1024 rows of 128256 with 20 alternatives 139 us.  With one mark for a warp, 64 alternatives
    // had nearly the whole row read again.)  Logits equal to the bar are let through unless it is a
    // mask's value (-inf or a type's lowest), of which there are too many.
    const uint32_t bar_key = sh.bar;
    bool strict = !(key_value(bar_key) > -3e38f), slow = false;   // (an empty bar, 0, lets everything through)
    for (;;) {
      const float bar = bar_key == 0 ? __int_as_float(0x7fffffff) : key_value(strict ? bar_key : key_below(bar_key));
      if (end_at >= 0 && !(end <= bar)) push(sh, end, end_at);
      uint32_t look = 0;   // the stretches to look through: each lane's own, all lanes at a time
      for (int mark = 0; mark << shift < rounds; ++mark)
        look |= !(__bfloat162float(sh.marks[mark][threadIdx.x]) <= bar) ? 1u << mark : 0;
      for (; look && *const_cast<volatile int*>(&sh.n_pushed) <= kPushed; look &= look - 1) {
        const int mark = __ffs(look) - 1;
#pragma unroll 1
        for (int round = mark << shift; round < min(rounds, (mark + 1) << shift); ++round) {
          const int at = mine0 + round * kStep;
          Vec<T> v[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u)
            if (at + u * kThreads < v1) {
              if (rounds <= kStages) v[u] = queue[round * kStep + u * kThreads];
              else v[u].v = body[at + u * kThreads];
            }
#pragma unroll
          for (int u = 0; u < kUnroll; ++u)
            if (at + u * kThreads < v1 && !(v[u].largest() <= bar))
#pragma unroll
              for (int i = 0; i < N; ++i)
                if (!(v[u][i] <= bar)) push(sh, v[u][i], pre + (at + u * kThreads) * N + i);
        }
      }
      __syncthreads();
      slow = sh.n_pushed > kPushed;
      if (!slow || strict) break;
      // long ties: without them
      strict = true;
      __syncthreads();
      if (threadIdx.x == 0) sh.n_pushed = 0;
      __syncthreads();
    }
    if (!slow) {
      const int above = sh.n_pushed;
      rank_list(sh.pushed, above, want, out);
      // those equal to a strict bar are not listed: the first of them fill what is missing
      for (int base = lo, have = above; have < want && base < hi; base += kThreads) {
        const int i = base + threadIdx.x;
        const bool same = i < hi && order_key(static_cast<float>(x[i])) == bar_key;
        const uint32_t votes = __ballot_sync(~0u, same);
        if (lane == 0) sh.warp_counts[warp] = __popc(votes);
        __syncthreads();
        int at = have + __popc(votes & ((1u << lane) - 1)), found = 0;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) at += sh.warp_counts[w];
          found += sh.warp_counts[w];
        }
        if (same && at < want) out[at] = place(static_cast<float>(x[i]), i);
        have += found;
        __syncthreads();
      }
    } else {
      // more than are ranked even so (NaN, or large logits that all fall to few groups): one search of the part for each
      unsigned long long last = ~0ull;
      for (int k = 0; k < want; ++k) {
        unsigned long long b = 0;
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
          const unsigned long long c = place(static_cast<float>(x[i]), i);
          if (c < last && c > b) b = c;
        }
        for (int o = 16; o; o >>= 1) {
          const unsigned long long c = __shfl_xor_sync(~0u, b, o);
          b = c > b ? c : b;
        }
        if (lane == 0) sh.best[warp] = b;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) b = sh.best[w] > b ? sh.best[w] : b;
        last = b;
        if (threadIdx.x == 0) out[k] = b;
        __syncthreads();
      }
    }
    __syncthreads();
  }

  // ---- the parts joined by the first of them
  if (parts > 1) {
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (part != 0) {
      uint32_t leader;
      const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(&sh));
      asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(leader) : "r"(here));
      const auto at = [&](const void* p) { return leader + static_cast<uint32_t>(__cvta_generic_to_shared(p)) - here; };
      if (threadIdx.x < static_cast<unsigned>(top_k)) {
        const unsigned long long p = static_cast<int>(threadIdx.x) < want ? out[threadIdx.x] : 0;
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at(&sh.lists[part][threadIdx.x])), "l"(p) : "memory");
      }
      if (threadIdx.x == kThreads - 1) {
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at(&sh.stats[part].m)), "f"(all.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at(&sh.stats[part].s)), "f"(all.s) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at(&sh.stats[part].t)), "f"(all.t) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at(&sh.befores[part])), "r"(before) : "memory");
      }
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (part != 0) return;
  }
  if (warp == kWarps - 1) {
    for (int p = 1; p < parts; ++p) {
      all = join(all, sh.stats[p]);
      before += sh.befores[p];
    }
    const float nan = __int_as_float(0x7fffffff), log_s = log1pf(all.s);
    const bool undefined = all.t != all.t || all.m == INFINITY, none = all.m == -INFINITY;
    if (lane == 0) {
      logprob[r] = undefined || !valid ? nan : none ? -INFINITY : (mine - all.m) - log_s;
      if (entropy) entropy[r] = undefined ? nan : none ? 0.f : log_s - all.t / (1.f + all.s);
      if (rank) rank[r] = valid ? before : -1;
      sh.stats[0] = {all.m, undefined ? nan : log_s, 0.f};
    }
  }
  if (top_k == 0) return;
  const unsigned long long* list = out;
  if (parts > 1) {
    // each part's list is in order: with its first `deep` entries no smaller than the least of
    // their last, top_k entries are, and whatever is smaller than that is out
    if (static_cast<int>(threadIdx.x) >= want && static_cast<int>(threadIdx.x) < top_k) out[threadIdx.x] = 0;   // (a short part)
    if (threadIdx.x == 0) sh.n_pushed = 0;
    __syncthreads();
    const int deep = (top_k + parts - 1) / parts;
    unsigned long long least = ~0ull;
    for (int p = 0; p < parts; ++p) least = min(least, sh.lists[p][deep - 1]);
    for (int i = threadIdx.x; i < parts * top_k; i += kThreads) {
      const unsigned long long c = sh.lists[i / top_k][i % top_k];
      if (c && c >= least) sh.pushed[atomicAdd(&sh.n_pushed, 1)] = c;
    }
    __syncthreads();
    const int n = sh.n_pushed;
    __syncthreads();
    rank_list(sh.pushed, n, top_k, sh.lists[1]);   // (all lists have been read)
    list = sh.lists[1];
  }
  __syncthreads();
  const float m = sh.stats[0].m, log_s = sh.stats[0].s;
  for (int k = threadIdx.x; k < top_k; k += kThreads) {
    const float v = key_value(static_cast<uint32_t>(list[k] >> 32));
    top_ids[r * top_k + k] = place_index(list[k]);
    top_logprobs[r * top_k + k] = log_s != log_s ? log_s : m == -INFINITY ? -INFINITY : (v - m) - log_s;
  }
}

template <class T>
xlpk_status launch(const T* logits, long long rows, int vocab, long long stride, const int* tokens, int top_k, float* logprob,
                   float* entropy, int* rank, int* top_ids, float* top_logprobs, int sms, cudaStream_t st) {
  // Parts keep the GPU busy while a thread still has two vectors or more: a row of 32000 takes 6.7 us
  // whole and 4.4 in 8 parts (fp32, no alternatives), 64 rows of 128256 20.5 whole, 11.8 in 4, 14.9 in
  // 8 (they no longer fit at once), 1024 rows 92.6 whole and 108 in 4.
  int parts = 1;
  while (parts < kMaxCluster && rows * parts * 2 <= 3 * sms && vocab / (parts * 2) >= 2 * kThreads * Vec<T>::N) parts *= 2;
  static std::atomic<unsigned long long> ready;   // devices whose kernel has its attributes
  int dev = 0;
  XLPK_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    XLPK_CUDA(cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared) + kQueueBytes));
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(rows * parts));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = sizeof(Shared) + kQueueBytes;
  c.stream = st;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = parts;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  c.attrs = &cluster;
  c.numAttrs = 1;
  XLPK_CUDA(cudaLaunchKernelEx(&c, logprobs_kernel<T>, logits, vocab, stride, tokens, top_k, parts, logprob, entropy,
                               rank, top_ids, top_logprobs));
  return XLPK_OK;
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
  if (vocab > 1 << 30) return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_token_logprobs: a vocabulary over 2^30");
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == XLPK_DTYPE_FP32)
    return launch(static_cast<const float*>(logits_dev), rows, vocab, row_stride, tokens_dev, top_k, logprob_dev, entropy_dev,
                  rank_dev, top_ids_dev, top_logprobs_dev, sms, st);
  return launch(static_cast<const __nv_bfloat16*>(logits_dev), rows, vocab, row_stride, tokens_dev, top_k, logprob_dev,
                entropy_dev, rank_dev, top_ids_dev, top_logprobs_dev, sms, st);
}
