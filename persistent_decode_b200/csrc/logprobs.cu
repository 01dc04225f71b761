// xlpk_token_logprobs: log probability, rank, entropy and top alternatives of
// given tokens under rows of logits (include/xlpk.h has the definition).
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
constexpr int kMaxCluster = 16;
constexpr int kGroups = 128;       // groups of threads, each known by its largest logit
constexpr int kPushed = 2048;     // candidates that fit while the row streams by
constexpr int kRanked = 1024;     // candidates that fit at the end
constexpr float kLog2e = 1.4426950408889634f;

// A logit's place in descending order: larger keys come first, NaN before +inf,
// -0 equals +0; ties go to the lower index.  No value has key 0.
__device__ inline uint32_t order_key(float x) {
  if (x != x) return 0xfffffffeu;   // (its bits without the sign are a NaN's again)
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
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
__device__ inline float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ inline float warp_sum(float x) {
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// Softmax statistics of a set of logits: the maximum m, and of all others (the
// maximum itself counts 1 and 0, exactly) s = sum e^(x-m), t = sum e^(x-m) (x-m).
// The others are kept apart so that log(1 + s) keeps a small s.
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
  static constexpr int U = sizeof(T) == 4 ? 4 : 2;   // vectors of a round: 16 logits; the next round's are in flight meanwhile
  uint4 v;
  __device__ float operator[](int i) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

// What one thread gathers of its part of a row.
struct Gather {
  float m = -INFINITY, s = 0.f, t = 0.f;   // m is the warp's; s and t of logits below it
  int ties = 0;                            // logits equal to m
  int before = 0;                          // logits that come before the token's
};

struct Shared {
  unsigned long long pushed[kPushed], ranked[kRanked];
  unsigned long long lists[kMaxCluster][kMaxTop];   // the leader's: every part's top tokens
  Stat stats[kMaxCluster];
  int befores[kMaxCluster];
  uint32_t groups[kGroups];                         // largest key of each group
  uint32_t bar;                                     // key: at least top_k + 1 groups have a larger one or this
  Stat warp_stats[kWarps];
  int warp_befores[kWarps], warp_counts[kWarps];
  unsigned long long best[kWarps];
  int n_pushed, n_ranked;
};

// Raises the bar to the (top_k + 1)-th largest of the groups' keys.  Keys only rise while
// this reads them, so whatever it finds is a bar that held at some time, and one that held
// once holds for good: top_k logits are at least that large, and ties are looked after at
// the end.  Threads 0 .. kGroups - 1 call it.
__device__ inline void raise_bar(Shared& sh, int top_k) {
  const volatile uint32_t* g = sh.groups;
  const uint32_t mine = g[threadIdx.x];
  int at_least = 0;
#pragma unroll 8
  for (int i = 0; i < kGroups; ++i) at_least += g[i] >= mine;
  if (at_least > top_k && mine > sh.bar) atomicMax(&sh.bar, mine);
}
// What a logit must not be <= to be pushed (NaN: everything is).
__device__ inline float bar_of(uint32_t key) { return key ? key_value(key) : __int_as_float(0x7fffffff); }

// Statistics and rank of one round: U vectors of each thread (FULL: all of them are there).
// Returns the thread's largest logit.
template <class T, bool FULL>
__device__ inline float round_stats(Gather& g, const Vec<T> (&v)[Vec<T>::U], int first, int there, int tok_vec, float bar_ge,
                                    float bar_gt) {
  constexpr int N = Vec<T>::N;
  float mine = -INFINITY;
#pragma unroll
  for (int u = 0; u < Vec<T>::U; ++u)
    if (FULL || u < there)
#pragma unroll
      for (int i = 0; i < N; ++i) mine = fmaxf(mine, v[u][i]);
  const float top = warp_max(mine);
  if (top >= g.m) {
    if (top > g.m) {
      const float d = g.m - top, w = ex2(d * kLog2e), all = g.s + g.ties;
      g.t = w > 0.f ? w * (g.t + d * all) : w * g.t;   // (d may be -inf)
      g.s = w * all;
      g.ties = 0;
      g.m = top;
    }
    // the maximum stands here: its ties are counted, not added
#pragma unroll
    for (int u = 0; u < Vec<T>::U; ++u)
      if (FULL || u < there)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float x = v[u][i];
          if (top == -INFINITY) {
            if (x != x) g.t = x;
          } else {
            const float d = max_nan(x - top, -1000.f), e = ex2(d * kLog2e);
            if (x < top) g.s += e;
            else ++g.ties;
            g.t += e * d;
          }
        }
  } else {
#pragma unroll
    for (int u = 0; u < Vec<T>::U; ++u)
      if (FULL || u < there)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float d = max_nan(v[u][i] - g.m, -1000.f), e = ex2(d * kLog2e);   // (e * d is 0 for -inf too)
          g.s += e;
          g.t += e * d;
        }
  }
#pragma unroll
  for (int u = 0; u < Vec<T>::U; ++u)
    if (FULL || u < there) {
      const float bar = first + u * kThreads < tok_vec ? bar_ge : bar_gt;
#pragma unroll
      for (int i = 0; i < N; ++i) g.before += !(v[u][i] <= bar);
    }
  return mine;
}

// Pushes the round's logits that the bar lets through (all lanes of a warp call it).
template <class T>
__device__ inline void push(const Vec<T> (&v)[Vec<T>::U], int first, int there, int pre, float bar, Shared& sh) {
  constexpr int N = Vec<T>::N;
  int n = 0;
#pragma unroll
  for (int u = 0; u < Vec<T>::U; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) n += u < there && !(v[u][i] <= bar);
  // one reservation for the warp
  const int lane = threadIdx.x & 31;
  int at = n;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, at, o);
    if (lane >= o) at += y;
  }
  int base = 0;
  if (lane == 31) base = atomicAdd(&sh.n_pushed, at);
  at += __shfl_sync(~0u, base, 31) - n;
  if (n == 0) return;
#pragma unroll
  for (int u = 0; u < Vec<T>::U; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (u < there && !(v[u][i] <= bar)) {
        if (at < kPushed) sh.pushed[at] = place(v[u][i], pre + (first + u * kThreads) * N + i);
        ++at;
      }
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

// The same for `parts` lists of top_k in descending order, by a search in each.
__device__ inline void rank_sorted(const unsigned long long (&lists)[kMaxCluster][kMaxTop], int parts, int top_k,
                                   unsigned long long* out) {
  for (int i = threadIdx.x; i < parts * top_k; i += kThreads) {
    const int p = i / top_k, k = i - p * top_k;
    const unsigned long long mine = lists[p][k];
    int r = k;
    for (int q = 0; q < parts && r < top_k; ++q) {
      if (q == p) continue;
      int lo = 0, hi = top_k;   // the first that is not larger
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (lists[q][mid] > mine) lo = mid + 1;
        else hi = mid;
      }
      r += lo;
    }
    if (r < top_k && mine) out[r] = mine;   // (place 0 fills up a part that is shorter than top_k)
  }
}

// One cluster per row, its CTAs taking consecutive parts.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const T* logits, int vocab, long long stride, const int* tokens,
                                                               int top_k, int parts, float* logprob,
                                                               float* entropy, int* rank, int* top_ids,
                                                               float* top_logprobs) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  constexpr int N = Vec<T>::N;
  const long long r = blockIdx.x / parts;
  const int part = blockIdx.x - static_cast<int>(r) * parts;
  const T* x = logits + r * stride;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // this CTA runs: its memory may be written
  // whole vectors of the row are [pre, pre + N * vecs); what is left at its ends goes to the first and last part
  const int pre = min(vocab, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
  const int vecs = (vocab - pre) / N, v0 = static_cast<int>(static_cast<long long>(vecs) * part / parts),
            v1 = static_cast<int>(static_cast<long long>(vecs) * (part + 1) / parts);
  const uint4* body = reinterpret_cast<const uint4*>(x + pre);

  Vec<T> v[Vec<T>::U], next[Vec<T>::U];
  const auto load = [&](Vec<T>(&to)[Vec<T>::U], int from) {
#pragma unroll
    for (int u = 0; u < Vec<T>::U; ++u)
      if (from + u * kThreads < v1) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(to[u].v.x), "=r"(to[u].v.y), "=r"(to[u].v.z), "=r"(to[u].v.w)
                     : "l"(body + from + u * kThreads));
      }
  };
  constexpr int kStep = Vec<T>::U * kThreads;
  int first = v0 + threadIdx.x;
  load(v, first);
  load(next, first + kStep);
  const int tok = tokens[r];
  const bool valid = tok >= 0 && tok < vocab;
  const float mine = valid ? static_cast<float>(x[tok]) : 0.f;
  if (threadIdx.x < kGroups) sh.groups[threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.n_pushed = sh.n_ranked = 0, sh.bar = 0;
  __syncthreads();

  // A logit comes before the token's if it is not <= gt, or, to the left of the token, not <= ge: the
  // float below the token's (NaN, and so everything, if there is none).  tok_vec: the vectors wholly to the left.
  const int tok_vec = tok < pre ? 0 : (tok - pre) / N;
  const uint32_t my_key = order_key(mine);
  const float bar_gt = mine, bar_ge = mine == -INFINITY ? __int_as_float(0x7fffffff)
                                                        : key_value(my_key - (my_key == 0x80000000u ? 2 : 1));   // (no -0)

  // the ends, one logit of a thread at most
  Gather g;
  int end_at = -1;
  if (part == 0 && static_cast<int>(threadIdx.x) < pre) end_at = threadIdx.x;
  if (part == parts - 1 && static_cast<int>(threadIdx.x) >= 32 && pre + vecs * N + static_cast<int>(threadIdx.x) - 32 < vocab)
    end_at = pre + vecs * N + threadIdx.x - 32;
  if (warp < 2) {
    const float e = end_at >= 0 ? static_cast<float>(x[end_at]) : -INFINITY;
    g.m = warp_max(e);
    if (end_at >= 0) {
      if (e != e) g.t = e;
      else if (g.m > -INFINITY) {
        const float d = fmaxf(e - g.m, -1000.f), w = ex2(d * kLog2e);
        if (e < g.m) g.s = w;
        else g.ties = 1;
        g.t = e == g.m ? e - e : w * d;   // (+inf: NaN)
      }
      g.before = !(e <= (end_at < tok ? bar_ge : bar_gt));
      if (top_k > 0) {
        atomicMax(&sh.groups[threadIdx.x % kGroups], order_key(e));
        const int at = atomicAdd(&sh.n_pushed, 1);
        sh.pushed[at] = place(e, end_at);   // at most 14
      }
    }
  }

  // ---- the row streams by
  int round = 0;
  const auto take = [&](const Vec<T>(&now)[Vec<T>::U]) {
    const int there = min(Vec<T>::U, max(0, (v1 - first + kThreads - 1) / kThreads));
    const float top = __all_sync(~0u, there == Vec<T>::U) ? round_stats<T, true>(g, now, first, there, tok_vec, bar_ge, bar_gt)
                                                        : round_stats<T, false>(g, now, first, there, tok_vec, bar_ge, bar_gt);
    if (top_k > 0) {
      // a thread below the bar has nothing that could raise it
      if (there > 0 && !(top <= bar_of(*const_cast<volatile uint32_t*>(&sh.bar))))
        atomicMax(&sh.groups[threadIdx.x % kGroups], order_key(top));
      if (round == 0) __syncthreads();   // every group has its first logit
      // (each time the row seen so far has doubled)
      if ((round & (round + 1)) == 0 && threadIdx.x < kGroups) raise_bar(sh, top_k);
      if (round == 0) __syncthreads();
      const float bar = bar_of(*const_cast<volatile uint32_t*>(&sh.bar));
      // a NaN is pushed whatever the maximum
      if (__any_sync(~0u, !(top <= bar) || g.t != g.t)) push(now, first, there, pre, bar, sh);
    }
    ++round;
    first += kStep;
  };
  for (int base = v0;;) {
    take(v);
    load(v, first + kStep);
    if ((base += kStep) >= v1) break;
    take(next);
    load(next, first + kStep);
    if ((base += kStep) >= v1) break;
  }
  if (top_k > 0) {
    __syncthreads();
    if (threadIdx.x < kGroups) raise_bar(sh, top_k);
  }

  // ---- this part's statistics
  {
    const float s = warp_sum(g.s), t = warp_sum(g.t);
    const int ties = __reduce_add_sync(~0u, g.ties), before = __reduce_add_sync(~0u, g.before);
    if (lane == 0) {
      sh.warp_stats[warp] = {g.m, s + (ties - 1), t};
      if (g.m == -INFINITY) sh.warp_stats[warp].s = 0.f;
      sh.warp_befores[warp] = before;
    }
  }
  __syncthreads();
  Stat all = sh.warp_stats[0];
  int before = 0;
  if (warp == 0) {
    // joined in the order of the warps
    for (int w = 1; w < kWarps; ++w) all = join(all, sh.warp_stats[w]);
    before = __reduce_add_sync(~0u, lane < kWarps ? sh.warp_befores[lane] : 0);
    if (valid && mine != mine) {
      // a NaN's rank: the NaN to its left
      before = 0;
      const int lo = part == 0 ? 0 : pre + v0 * N, hi = part == parts - 1 ? vocab : pre + v1 * N;
      for (int i = lo + lane; i < min(hi, tok); i += 32) before += order_key(static_cast<float>(x[i])) == my_key;
      before = __reduce_add_sync(~0u, before);
    } else if (valid && tok >= pre && tok_vec >= v0 && tok_vec < v1) {
      // equals to the left of the token in its own vector
      const int i = pre + tok_vec * N + lane;
      before += __reduce_add_sync(~0u, static_cast<int>(i < tok && static_cast<float>(x[min(i, tok)]) == mine));
    }
  }

  // ---- this part's top tokens, in order
  const int lo = part == 0 ? 0 : pre + v0 * N, hi = part == parts - 1 ? vocab : pre + v1 * N;
  const int want = min(top_k, hi - lo);
  unsigned long long* const out = sh.lists[0];
  if (top_k > 0) {
    const uint32_t least = sh.bar;
    const int n = sh.n_pushed;
    bool slow = n > kPushed;
    if (!slow) {
      for (int i = threadIdx.x; i < n; i += kThreads)
        if (static_cast<uint32_t>(sh.pushed[i] >> 32) > least) {
          const int at = atomicAdd(&sh.n_ranked, 1);
          if (at < kRanked) sh.ranked[at] = sh.pushed[i];
        }
      __syncthreads();
      slow = sh.n_ranked > kRanked;
    }
    if (!slow) {
      const int above = sh.n_ranked;
      rank_list(sh.ranked, above, want, out);
      // logits equal to the bar (masked rows, long ties) are not pushed: the first of them fill what is missing
      for (int base = lo, have = above; have < want && base < hi; base += kThreads) {
        const int i = base + threadIdx.x;
        const bool same = i < hi && order_key(static_cast<float>(x[i])) == least;
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
      // more candidates than fit (rows in rising order, or of NaN): one search of the part for each
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
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (part != 0) {
      uint32_t leader;
      const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(&sh));
      asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(leader) : "r"(here));
      const auto at = [&](const void* p) { return leader + static_cast<uint32_t>(__cvta_generic_to_shared(p)) - here; };
      if (threadIdx.x < static_cast<unsigned>(top_k)) {
        const unsigned long long p = static_cast<int>(threadIdx.x) < want ? out[threadIdx.x] : 0;
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at(&sh.lists[part][threadIdx.x])), "l"(p) : "memory");
      }
      if (threadIdx.x == 0) {
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at(&sh.stats[part].m)), "f"(all.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at(&sh.stats[part].s)), "f"(all.s) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at(&sh.stats[part].t)), "f"(all.t) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at(&sh.befores[part])), "r"(before) : "memory");
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (part != 0) return;
  }
  if (warp == 0) {
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
  if (parts > 1) {
    if (static_cast<int>(threadIdx.x) >= want && static_cast<int>(threadIdx.x) < top_k) out[threadIdx.x] = 0;
    __syncthreads();
    rank_sorted(sh.lists, parts, top_k, sh.ranked);
  }
  __syncthreads();
  const unsigned long long* const list = parts > 1 ? sh.ranked : out;
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
  int parts = 1;
  while (parts < kMaxCluster && rows * parts * 2 <= 4 * sms && vocab / (parts * 2) >= kThreads * Vec<T>::N) parts *= 2;
  static std::atomic<unsigned long long> ready;   // devices whose kernel has its attributes
  int dev = 0;
  XLPK_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    XLPK_CUDA(cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    XLPK_CUDA(cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared)));
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(rows * parts));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = sizeof(Shared);
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
