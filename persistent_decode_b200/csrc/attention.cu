// xlpk_decode_attention: attention of one new token per sequence over its KV
// cache (include/xlpk.h has the definition).
//
// Mathematics.  Over the visible positions t in any order and grouping, with
// running m = max s_t, l = sum 2^(s_t - m), o = sum 2^(s_t - m) v_t (s in units
// of log 2): two groups join as m = max(m1, m2), l = l1 2^(m1-m) + l2 2^(m2-m),
// o alike; out = o / l, lse = (m + log2 l) ln 2.  A tile is 16 positions; a warp
// takes two at a time, keeps m, l and o of up to 16 query heads in registers and
// joins with others only where its stretch of a segment (one kv head of one
// sequence) ends.
//
// Bound.  Each K and V entry is read once and meets n_q / n_kv query heads: 4 to
// 14 flop a byte, far below the tensor cores' ridge, so the floor is the cache's
// bytes at HBM rate.  (Times: of a captured call replayed, on the device; among
// calls through Python they are 3 to 22 us longer.)  One long sequence comes to
// 91% of the copy rate (131072 positions of 8 kv heads of 128, bf16: 91 us for
// 537 MB).  What keeps shorter ones from it is fixed: about 4 us from launch to
// the first data and 3.5 us for the join.  e4m3 halves the bytes and not the work:
// each code is widened to fp16 by a conversion, and a tile of 4 KB takes 341
// instructions.  They are issued in 37% of cycles, with the tensor pipe active in
// 28%: the loop waits for its own chain of scores, softmax and p v, with two warps
// a scheduler, and runs at 71% of the copy rate (four of 131072, d 128: 235 us for
// 1.07 GB).
//
// Precision.  m16n8k16 MMAs with fp32 sums, which are added up rounded every FOLD
// tiles (they cut off).  Cache entries are exact operands (bf16, or e4m3 widened to
// fp16); q and p are split into as many 16-bit terms as their type needs: one for
// a bf16 q, three of bf16 or two of fp16 for an fp32 q, two (three with fp32
// output) for p, so that p's rounding stays far below the output's.  In fp16,
// weights below 2^-34 of a tile's largest vanish.  With up to 8 heads a group the
// second term sits in rows 8-15 of the A operand and costs no MMA.  The scores
// never leave registers: the C fragment of q.k is the A fragment of p.v.
//
// Layout.  A K row is multiplied through a permutation of its dims that lets a
// lane's 16 bytes of it be its B fragments as they are; likewise e4m3 V.  So a
// lane reads only what it copied itself (cp.async, a queue of 16-byte chunks in
// shared memory) and the loop has no barrier.  bf16 V goes through ldmatrix.trans
// instead, which spares the byte permutation of each pair of its rows.
//
// Why mma.sync: a tile's contraction is 4 to 16 query rows wide; tcgen05 starts
// at 64 rows and keeps sums in tensor memory, from which the scores would have
// to come back for the softmax.  The tensor pipe is active a quarter of the time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/xlpk.h"
#include "errors.h"

using namespace xlpk;

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFarScore = 0x1p22f;   // in powers of 2: fp32's step is half of one
constexpr int kJoinWarps = 8;
constexpr int kThreads = kJoinWarps * 32;   // of the join
constexpr int kMaxCtas = 160;               // one for each SM
constexpr int kPieces = 4;                  // that warps as workers may cut a segment into, about
constexpr int kTile = 16;   // positions of a tile; a warp takes two of its tiles at a time

struct Args {
  xlpk_attention_args a;
  float* parts;     // [workers][2] slots of partial results
  int ctas;         // of the attention
  float s2;         // scale * log2(e); for an e4m3 cache s2 * 2^exp is that times k_scale, s2 in [0.5, 1]
  int exp;
  int page_shift;   // log2 of page_size, or -1
  bool flat;        // the visible rows of a tile are in one page
  int4* joins;      // [workers] (sequence, kv head, last worker, -) of the segment that a worker begins and another ends; .x < 0: none
  int* team;        // warps of a worker
};

// The tiles of one sequence: those that hold a visible position.
struct Seq {
  int n;       // positions
  int lo;      // the window's first position; the first tokens before it are visible too
  int head;    // tiles of first tokens, before the gap
  int skip;    // tiles of the gap
  int tiles;   // all but the gap's
};
__device__ inline Seq seq_of(const xlpk_attention_args& a, int b) {
  Seq s;
  s.n = a.seq_lens_dev[b];
  if (s.n < 0 || s.n > static_cast<long long>(a.table_cols) * a.page_size) s.n = 0;
  s.lo = a.window > 0 && s.n > a.window ? s.n - a.window : 0;
  s.head = (min(a.sinks, s.lo) + kTile - 1) / kTile;
  s.skip = max(s.lo / kTile - s.head, 0);
  s.tiles = (s.n + kTile - 1) / kTile - s.skip;
  return s;
}
__device__ inline int tile_pos(const Seq& s, int i) { return (i < s.head ? i : i + s.skip) * kTile; }
__device__ inline bool visible(const xlpk_attention_args& a, const Seq& s, int t) {
  return t < s.n && (t >= s.lo || t < a.sinks);
}

// One stretch of consecutive tiles in the order (sequence, kv head, tile), cut
// at segment borders: a segment is one kv head of one sequence.
struct Walk {
  int b, h, i, end;      // tiles [i, end) of segment (b, h)
  int left;              // tiles after them
  Seq s;
};
__device__ inline void walk_cut(Walk& w, int n) {
  w.end = w.i + min(n, w.s.tiles - w.i);
  w.left = n - (w.end - w.i);
}
// To the next segment (left > 0).
__device__ inline void walk_next(const xlpk_attention_args& a, Walk& w) {
  if (++w.h == a.n_kv_heads) {
    w.h = 0;
    do w.s = seq_of(a, ++w.b);
    while (w.s.tiles == 0);
  }
  w.i = 0;
  walk_cut(w, w.left);
}

// `total` tiles over `workers`, the first `more` of which take one more than the others.
struct Shares {
  unsigned each, more;
  __device__ Shares(unsigned total, unsigned workers) : each(total / workers), more(total - each * workers) {}
  __device__ int first(int worker) const { return worker * each + min(static_cast<unsigned>(worker), more); }
  __device__ int owner(unsigned tile) const {
    const unsigned split = more * (each + 1);
    return tile < split ? tile / (each + 1) : more + (tile - split) / each;
  }
};

template <int D_, bool KV8_, bool WIDE_, bool IO32_>
struct Shape {
  static constexpr int D = D_;
  static constexpr bool KV8 = KV8_;      // e4m3 cache, fp16 operands; else bf16
  static constexpr bool WIDE = WIDE_;    // 9 to 16 query heads per kv head; else up to 8
  static constexpr bool IO32 = IO32_;
  // Eight warps have registers for four chains of MMAs.  e4m3 rows of 64 leave enough for twelve and
  // two chains (16 sequences of 8192, d 64: 8 warps 53 us, 12 46, 16 48; four of 131072, d 128: 8 warps
  // 233 us, 12, which spill, 246; all when this was chosen, 47 and 235 now).
  static constexpr int WARPS = !WIDE && KV8 && D == 64 ? 12 : 8, THREADS = WARPS * 32;
  static constexpr int CHAINS = WARPS == 8 ? 4 : 2;   // scores' chains of MMAs that run at once
  static constexpr int E = KV8 ? 1 : 2;
  static constexpr int ROWS = WIDE ? 16 : 8;
  // what one lane copies of a cache row: a K row is read by the 4 lanes of a quad in 16-byte
  // chunks, a V row by the 8 lanes that share a quad position
  static constexpr int KC = D * E / 64;
  static constexpr int VB = D * E / 8 >= 16 ? 16 : 8;
  static constexpr int VC = D * E / 8 / VB;
  static constexpr int KBYTES = 2 * KC * 512, STAGE = KBYTES + 4 * VC * VB * 32;
  static constexpr int MERGE = WARPS * ROWS * (D + 2) * 4;
  static constexpr int FIT = (232448 - 1024 - MERGE) / (STAGE * WARPS);
  static constexpr int STAGES = FIT < 8 ? FIT : 8;
  static constexpr int SMEM = STAGES * STAGE * WARPS + MERGE;
  static_assert(STAGES >= 2, "a step takes two tiles");
  static constexpr int QT = IO32 ? (KV8 ? 2 : 3) : 1;   // terms of q
  static constexpr int PT = IO32 && !KV8 ? 3 : 2;       // terms of p
  static constexpr int QR = D / 8;                      // registers of one term of one row
  static constexpr bool LOW = WIDE && QT > 1;           // the lower terms' scores have sums of their own (else: rows 8-15)
  static constexpr float SHIFT = KV8 ? 10.f : 0.f;      // p is held times 2^SHIFT: fp16 has 2^-14 for its lower term then
  static constexpr int SLOT = ROWS * (D + 2);           // floats of a partial result
  static constexpr int FOLD = WIDE ? 32 : 64;           // tiles of a warp between additions to its sum in memory

  // Where the 4 dims from 4 c of a head stand in the merge scratch's row: swizzled so that lanes that write at the
  // same time (all t, and consecutive heads) do so in different banks.
  __device__ static int place(int head, int c) {
    if (!KV8) return (c ^ (head & 3) << 1) * 4;
    return (D == 128 ? c ^ (c >> 3 & 3) ^ (head & 1) << 2 : c ^ (c >> 3 & 1) ^ (head & 1) << 1) * 4;
  }
};

__device__ inline void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                           bool f16) {
  if (f16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The next 16-bit term of x and y as a register; x and y keep the remainders.
template <bool F16>
__device__ inline uint32_t term(float& x, float& y) {
  uint32_t r;
  if (F16) {
    const __half2 h = __floats2half2_rn(x, y);
    x -= __low2float(h), y -= __high2float(h);
    r = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    x -= __low2float(h), y -= __high2float(h);
    r = *reinterpret_cast<const uint32_t*>(&h);
  }
  return r;
}

// Two e4m3 codes (the low 16 bits) as two fp16 values, exactly.
__device__ inline uint32_t widen(uint32_t codes) {
  uint32_t r;
  asm("{ .reg .b16 l; mov.b32 {l, _}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(codes));
  return r;
}

__device__ inline uint32_t widen_high(uint32_t codes) {
  uint32_t r;
  asm("{ .reg .b16 h; mov.b32 {_, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(codes));
  return r;
}

template <bool IO32, int N>
__device__ inline void load_row(const void* base, long long at, float (&x)[N]) {
  if (IO32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 v = p[i];
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const uint4 v = p[i];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
}

template <bool IO32>
__device__ inline void store_out(void* base, long long at, float4 v) {
  if (IO32) {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = v;
  } else {
    const __nv_bfloat162 l = __floats2bfloat162_rn(v.x, v.y), h = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&l), *reinterpret_cast<const uint32_t*>(&h));
  }
}

// N elements of a new row as cache entries: `bytes` of them in w.
template <bool KV8, int N>
__device__ inline void round_row(const float (&x)[N], float inv_scale, uint32_t* w) {
  if (KV8) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv_scale, x[4 * i + 1] * inv_scale), __NV_SATFINITE, __NV_E4M3);
      const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv_scale, x[4 * i + 3] * inv_scale), __NV_SATFINITE, __NV_E4M3);
      w[i] = l | h << 16;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

template <int BYTES>
__device__ inline void copy_async(uint32_t dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// Zeros unless `real`; then nothing is read.
template <int BYTES>
__device__ inline void copy_async(uint32_t dst, const void* src, bool real) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(real ? 8 : 0) : "memory");
}

// -126 <= e <= 127
__device__ inline float power_of_2(int e) { return __int_as_float((e + 127) << 23); }

// 2^x to 2^-22, 0 for -inf.
__device__ inline float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ inline float lse_of(float m, float l) { return l == 0 ? -INFINITY : m * kLn2 + logf(l); }

template <class S>
__global__ void __launch_bounds__(S::THREADS, 1) attention_kernel(const __grid_constant__ Args args) {
  extern __shared__ __align__(128) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;");   // the join may be set up meanwhile; it waits for this grid's end
  __shared__ int scan[S::WARPS], most[S::WARPS], start[S::WARPS][2];
  const xlpk_attention_args& a = args.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int group = a.n_q_heads / a.n_kv_heads;
  constexpr int D = S::D;

  // ---- the worker's even share [x0, x0 + count) of all tiles, and the segment it begins in.
  // A worker is a CTA whose warps take a segment's tiles in turn, or, where that cuts no segment into
  // more than about kPieces, a warp: then a short segment costs no barrier and no idle warps (64
  // sequences of 1024, 8 kv heads: 35 us against 38 with CTAs).  Longer segments lose by it: their
  // pieces go through memory (64 behind a 4096 window: 101 us against 95).
  Walk w{};
  int count, x0;
  Shares shares(1, 1);
  int worker, workers, team;
  {
    const int per = (a.n_seqs + S::THREADS - 1) / S::THREADS, b0 = min(static_cast<int>(threadIdx.x) * per, a.n_seqs),
              b1 = min(b0 + per, a.n_seqs);
    int mine = 0, longest = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = seq_of(a, b).tiles;
      mine += n;
      longest = max(longest, n);
    }
    longest = __reduce_max_sync(~0u, longest);
    int sum = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) scan[warp] = sum, most[warp] = longest;
    __syncthreads();
    int total = 0, before = sum - mine;
#pragma unroll 1
    for (int i = 0; i < S::WARPS; ++i) {
      if (i < warp) before += scan[i];
      total += scan[i];
      longest = max(longest, most[i]);
    }
    total *= a.n_kv_heads;
    const int warps = gridDim.x * S::WARPS;
    team = static_cast<long long>(longest) * warps <= static_cast<long long>(kPieces) * total ? 1 : S::WARPS;
    const int all = team == 1 ? warps : gridDim.x;
    worker = team == 1 ? blockIdx.x * S::WARPS + warp : blockIdx.x;
    workers = min(total, all);
    if (workers > 0) shares = Shares(total, workers);
    if (mine > 0)
#pragma unroll 1
      for (int i = 0; i < S::WARPS / team; ++i) {
        const int wk = blockIdx.x * (S::WARPS / team) + i;
        if (wk >= workers) break;
        const int x = shares.first(wk);
        if (x < before * a.n_kv_heads || x >= (before + mine) * a.n_kv_heads) continue;
        int b = b0;
        int off = x - before * a.n_kv_heads;
        for (;; ++b) {
          const int seg = seq_of(a, b).tiles * a.n_kv_heads;
          if (off < seg) break;
          off -= seg;
        }
        start[i][0] = b;
        start[i][1] = off;
      }
    // who joins the pieces of the segment that this worker begins and does not end is said at its end
    if (lane == 0 && (team == 1 || warp == 0)) args.joins[worker] = make_int4(-1, 0, 0, 0);
    if (blockIdx.x == 0 && threadIdx.x == 0) *args.team = team;
    __syncthreads();
    const bool any = worker < workers;
    x0 = any ? shares.first(worker) : 0;
    count = any ? shares.first(worker + 1) - x0 : 0;
    if (any) {
      const int* at = start[team == 1 ? warp : 0];
      w.b = at[0];
      w.s = seq_of(a, w.b);
      w.h = static_cast<unsigned>(at[1]) / static_cast<unsigned>(w.s.tiles);
      w.i = at[1] - w.h * w.s.tiles;
      walk_cut(w, count);
    }
  }
  const int lead = team == 1 ? warp : 0, rank = warp - lead;   // the worker's first warp, and this one's place in it

  // ---- rows without positions
  for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
    const int n = a.seq_lens_dev[b];
    const bool bad = n < 0 || n > static_cast<long long>(a.table_cols) * a.page_size;
    if (n != 0 && !bad) continue;
    const float v = bad ? __int_as_float(0x7fffffff) : 0.f;
    for (int i = threadIdx.x * 4; i < a.n_q_heads * D; i += S::THREADS * 4)
      store_out<S::IO32>(a.out_dev, b * a.out_seq_stride + i / D * a.out_head_stride + i % D, make_float4(v, v, v, v));
    if (a.lse_dev)
      for (int i = threadIdx.x; i < a.n_q_heads; i += S::THREADS)
        a.lse_dev[static_cast<long long>(b) * a.n_q_heads + i] = bad ? v : -INFINITY;
    if (bad && a.status_dev && threadIdx.x == 0) *a.status_dev = XLPK_ERR_INVALID_ARG;
  }
  if (count == 0) return;

  // ---- the warp's queue of tiles in shared memory.  K, and e4m3 V, are read by the lane that
  // copied them; bf16 V is laid out in rows for ldmatrix, its 16-byte chunks swizzled.
  const uint32_t queue = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * S::STAGES * S::STAGE;
  const uint8_t* queue_at = smem + warp * S::STAGES * S::STAGE;
  // where this lane puts chunk c of V row 2t + (r & 1) + 8 (r >> 1)
  const auto v_slot = [&](int r, int c) {
    if (S::KV8) return S::KBYTES + ((r * S::VC + c) * 32 + lane) * S::VB;
    const int row = 2 * t + (r & 1) + (r >> 1) * 8;
    return S::KBYTES + row * D * 2 + (((c * 8 + g) ^ (row & 7)) & (D / 8 - 1)) * 16;
  };
  Walk f = w;            // the tile that is fetched next
  f.i += rank;
  int bad_stages = 0;
  bool more = true;
  // Pages are looked up ahead of the copies that need them.  Where a tile never crosses a page,
  // lane i holds the page of the i-th of the segment's next 32 tiles of this warp, and `later` those
  // of the 32 after them; otherwise every lane holds the page of one position of the next tile
  // (16..31 as 0..15).  -1: not visible, -2: outside the pool.
  int pages = -1, later = -1, used = 0;
  const auto page_of = [&](int pos) {
    const int j = args.page_shift >= 0 ? pos >> args.page_shift : pos / a.page_size;
    const int page = a.page_table_dev ? a.page_table_dev[f.b * a.table_stride + j] : f.b;
    return page < 0 || page >= a.n_pages ? -2 : page;
  };
  const auto in_page = [&](int pos) { return args.page_shift >= 0 ? pos & (a.page_size - 1) : pos % a.page_size; };
  const auto batch = [&](int i) { return i < f.end ? page_of(min(tile_pos(f.s, i), f.s.n - 1)) : -1; };
  const auto settle = [&](bool fresh) {   // to the next tile; `fresh`: of a segment that is new
    while (f.i >= f.end) {
      if (f.left == 0) {
        more = false;
        return;
      }
      walk_next(a, f);
      f.i += rank;
      fresh = true;
    }
    if (!args.flat) {
      const int pos = tile_pos(f.s, f.i) + (lane & 15);
      pages = visible(a, f.s, pos) ? page_of(pos) : -1;
    } else if (fresh) {
      pages = batch(f.i + lane * team);
      later = batch(f.i + (lane + 32) * team);
      used = 0;
    } else if (++used == 32) {
      pages = later;
      later = batch(f.i + (lane + 32) * team);
      used = 0;
    }
  };
  auto fetch = [&](int stage) {
    if (more) {
      const int pos = tile_pos(f.s, f.i);
      const int fresh = a.k_new_dev && f.i == f.s.tiles - 1 ? f.s.n - 1 - pos : -1;   // the row of the new token
      const uint32_t dst = queue + stage * S::STAGE;
      const int page = args.flat ? __shfl_sync(~0u, pages, used) : -1;
      if (page >= 0 && fresh < 0 && pos + kTile <= f.s.n && (pos >= f.s.lo || pos + kTile <= a.sinks)) {
        // 16 visible rows of one page
        bad_stages &= ~(1 << stage);
        const int in = in_page(pos);
        const long long kstep = a.k_pos_stride * S::E, vstep = a.v_pos_stride * S::E;
        const uint8_t* k = static_cast<const uint8_t*>(a.k_dev) +
                           (page * a.k_page_stride + in * a.k_pos_stride + f.h * a.k_head_stride) * S::E + g * kstep + t * 16;
        const uint8_t* v = static_cast<const uint8_t*>(a.v_dev) +
                           (page * a.v_page_stride + in * a.v_pos_stride + f.h * a.v_head_stride) * S::E + 2 * t * vstep + g * S::VB;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int j = 0; j < S::KC; ++j) copy_async<16>(dst + ((r * S::KC + j) * 32 + lane) * 16, k + j * 64);
          k += 8 * kstep;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
          for (int c = 0; c < S::VC; ++c) copy_async<S::VB>(dst + v_slot(r, c), v + c * 128);
          v += r == 1 ? 7 * vstep : vstep;
        }
      } else {
        const int at = pos + (lane & 15), in_f = in_page(at),
                  page_f = !args.flat ? pages : visible(a, f.s, at) ? page : -1;
        const bool bad = __any_sync(~0u, page_f == -2);
        bad_stages = bad ? bad_stages | 1 << stage : bad_stages & ~(1 << stage);
        const long long ko = page_f < 0 ? -1 : page_f * a.k_page_stride + in_f * a.k_pos_stride + f.h * a.k_head_stride;
        const long long vo = page_f < 0 ? -1 : page_f * a.v_page_stride + in_f * a.v_pos_stride + f.h * a.v_head_stride;
        uint8_t* out = const_cast<uint8_t*>(queue_at) + stage * S::STAGE;
#pragma unroll 1
        for (int r = 0; r < 2; ++r) {
          const long long o = __shfl_sync(~0u, ko, g + 8 * r);
          uint8_t* row = static_cast<uint8_t*>(a.k_dev) + (o < 0 ? 0 : o * S::E);
          if (fresh == g + 8 * r) {
#pragma unroll
            for (int j = 0; j < S::KC; ++j) {
              constexpr int N = 16 / S::E;
              float x[N];
              uint32_t c[4];
              load_row<S::IO32>(a.k_new_dev, f.b * a.new_k_seq_stride + f.h * a.new_k_head_stride + j * 4 * N + t * N, x);
              round_row<S::KV8>(x, 1.f / a.k_scale, c);
              const uint4 v = make_uint4(c[0], c[1], c[2], c[3]);
              *reinterpret_cast<uint4*>(out + ((r * S::KC + j) * 32 + lane) * 16) = v;
              if (o >= 0) *reinterpret_cast<uint4*>(row + j * 64 + t * 16) = v;
            }
          } else {
#pragma unroll
            for (int j = 0; j < S::KC; ++j)
              copy_async<16>(dst + ((r * S::KC + j) * 32 + lane) * 16, row + j * 64 + t * 16, o >= 0);
          }
        }
#pragma unroll 1
        for (int r = 0; r < 4; ++r) {
          const int at = 2 * t + (r & 1) + (r >> 1) * 8;
          const long long o = __shfl_sync(~0u, vo, at);
          uint8_t* row = static_cast<uint8_t*>(a.v_dev) + (o < 0 ? 0 : o * S::E);
          if (fresh == at) {
#pragma unroll
            for (int c = 0; c < S::VC; ++c) {
              constexpr int N = 16 / S::E;   // (a lane of 8 codes rounds 16 and keeps its half)
              float x[N];
              uint32_t code[4];
              const int first = c * 128 / S::E + g * (S::VB / S::E);
              load_row<S::IO32>(a.v_new_dev, f.b * a.new_v_seq_stride + f.h * a.new_v_head_stride + first / N * N, x);
              round_row<S::KV8>(x, 1.f / a.v_scale, code);
              uint8_t* q = out + v_slot(r, c);
              if (S::VB == 16) {
                const uint4 v = make_uint4(code[0], code[1], code[2], code[3]);
                *reinterpret_cast<uint4*>(q) = v;
                if (o >= 0) *reinterpret_cast<uint4*>(row + c * 128 + g * 16) = v;
              } else {
                const uint2 v = first % N ? make_uint2(code[2], code[3]) : make_uint2(code[0], code[1]);
                *reinterpret_cast<uint2*>(q) = v;
                if (o >= 0) *reinterpret_cast<uint2*>(row + g * 8) = v;
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < S::VC; ++c) copy_async<S::VB>(dst + v_slot(r, c), row + c * 128 + g * S::VB, o >= 0);
          }
        }
        if (bad && a.status_dev && lane == 0) *a.status_dev = XLPK_ERR_INVALID_ARG;
      }
      f.i += team;
      settle(false);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  settle(true);
#pragma unroll 1
  for (int i = 0; i < S::STAGES; ++i) fetch(i);

  float* const merge = reinterpret_cast<float*>(smem + S::STAGES * S::STAGE * S::WARPS);
  float* const merge_m = merge + S::WARPS * S::ROWS * D;
  float* const merge_l = merge_m + S::WARPS * S::ROWS;
  const auto worker_sync = [&]() {
    if (team == 1) __syncwarp();
    else __syncthreads();
  };
  int x = x0;   // the segment's first tile here
  int stage = 0;
  for (;;) {
    // ---- q of the segment's heads, as terms
    uint32_t q[S::WIDE ? 2 : 1][S::QT][S::QR];
    float rs[S::WIDE ? 2 : 1];   // what makes powers of 2 of the row's scores (e4m3; else args.s2 does)
#pragma unroll
    for (int r = 0; r < (S::WIDE ? 2 : 1); ++r) {
      float v[D / 4];
      const int head = g + 8 * r;
      if (head < group) {
        constexpr int N = 16 / S::E;
#pragma unroll
        for (int j = 0; j < S::KC; ++j)
          load_row<S::IO32>(a.q_dev, w.b * a.q_seq_stride + (w.h * group + head) * a.q_head_stride + j * 4 * N + t * N,
                            *reinterpret_cast<float(*)[N]>(v + j * N));
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) v[i] = 0.f;
      }
      if (S::KV8) {
        // fp16 terms: the row is scaled by the power of two that brings its largest entry to
        // [2^10, 2^11): 11 bits of each entry and 11 of what they leave hold it to 2^-24 of itself, or to
        // 2^-35 of the largest.
        // (2^e alone may be out of range, and so may the scale's product with 2^-e before it is whole.)
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(v[i]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const int e = top > 0.f && top < INFINITY ? 10 - ilogbf(top) : 0;
        const float up = power_of_2(min(e, 100)), more_up = power_of_2(max(e - 100, 0));
#pragma unroll
        for (int i = 0; i < D / 4; ++i) v[i] *= up, v[i] *= more_up;
        const int down = min(max(args.exp - e, -252), 252), half = down / 2;
        // (neither infinity nor 0: scores of 0 stay 0, those of hidden positions -inf)
        rs[r] = fmaxf(fminf(args.s2 * power_of_2(half) * power_of_2(down - half), 0x1.fffffep127f), 0x1p-126f);
      }
#pragma unroll
      for (int i = 0; i < S::QR; ++i)
#pragma unroll
        for (int k = 0; k < S::QT; ++k) q[r][k][i] = term<S::KV8>(v[2 * i], v[2 * i + 1]);
    }

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool bad = false;
    int i = w.i + rank;

    // Sums of MMAs are cut off, not rounded, so over many tiles they fall behind (by 2.4e-5 to 5.4e-5 where a
    // warp sums up 590 to 886 tiles of positive values).  Every FOLD tiles a warp adds them to a sum in its scratch,
    // which is rounded.
#pragma unroll 1
    while (i < w.end) {
      float o[D / 8][4];
#pragma unroll
      for (int i2 = 0; i2 < D / 8; ++i2) o[i2][0] = o[i2][1] = o[i2][2] = o[i2][3] = 0.f;
      const int stop = min(w.end, i + S::FOLD * team);
#pragma unroll 1
      for (; i < stop; i += 2 * team) {
        const bool pair = i + team < w.end;
        asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 2) : "memory");
        __syncwarp();   // V was copied by other lanes too
        const int stage2 = stage + 1 == S::STAGES ? 0 : stage + 1;
        // ---- scores: positions are the columns, two tiles side by side, so that four chains of MMAs
        // run at once.  (Where there is no second tile, what is in its slot is multiplied and masked.)
        float s[4][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        float low[S::LOW ? 4 : 1][4] = {};   // what the lower terms add: each sum loses its own last bits only
#pragma unroll
        for (int n0 = 0; n0 < 4; n0 += S::CHAINS)
#pragma unroll
        for (int j = 0; j < S::KC; ++j) {
          constexpr int NB = S::KV8 ? 8 : 4;
          uint32_t kb[S::CHAINS][NB];
#pragma unroll
          for (int i = 0; i < S::CHAINS; ++i) {
            const int nt = n0 + i;
            const uint4 k4 = *reinterpret_cast<const uint4*>(queue_at + (nt >> 1 ? stage2 : stage) * S::STAGE +
                                                             (((nt & 1) * S::KC + j) * 32 + lane) * 16);
            const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) {
              if (S::KV8)
                kb[i][(2 * i2) % NB] = widen(kw[i2]), kb[i][(2 * i2 + 1) % NB] = widen_high(kw[i2]);
              else
                kb[i][i2] = kw[i2];
            }
          }
#pragma unroll
          for (int p = 0; p < NB; p += 2) {
            const int c = j * NB + p;
#pragma unroll
            for (int k = 0; k < (S::WIDE ? S::QT : (S::QT + 1) / 2); ++k)
#pragma unroll
              for (int i = 0; i < S::CHAINS; ++i) {
                float(&sc)[4] = s[n0 + i];
                if (S::WIDE)
                  mma(S::LOW && k > 0 ? low[(n0 + i) * S::LOW] : sc, q[0][k][c], q[S::WIDE][k][c], q[0][k][c + 1], q[S::WIDE][k][c + 1], kb[i][p], kb[i][p + 1], S::KV8);
                else if (2 * k + 1 < S::QT)
                  mma(sc, q[0][2 * k][c], q[0][(2 * k + 1) % S::QT][c], q[0][2 * k][c + 1], q[0][(2 * k + 1) % S::QT][c + 1],
                      kb[i][p], kb[i][p + 1], S::KV8);
                else
                  // (a third term joins the second)
                  mma(sc, S::QT > 1 ? 0 : q[0][2 * k][c], S::QT > 1 ? q[0][2 * k][c] : 0, S::QT > 1 ? 0 : q[0][2 * k][c + 1],
                      S::QT > 1 ? q[0][2 * k][c + 1] : 0, kb[i][p], kb[i][p + 1], S::KV8);
              }
          }
        }
        if (!S::WIDE && S::QT > 1)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) s[nt][0] += s[nt][2], s[nt][1] += s[nt][3];
        if (S::LOW)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[nt][c] += low[nt * S::LOW][c];
        // ---- online softmax over the two tiles
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int pos = tile_pos(w.s, i + half * team);
          if ((half && !pair) || pos + kTile > w.s.n || (pos < w.s.lo && pos + kTile > a.sinks)) {
#pragma unroll
            for (int n2 = 0; n2 < 2; ++n2)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if ((half && !pair) || !visible(a, w.s, pos + 8 * n2 + 2 * t + (c & 1))) s[half * 2 + n2][c] = -INFINITY;
          }
        }
        constexpr int NR = S::WIDE ? 2 : 1;
        uint32_t pt[NR][S::PT][4];
        bool grow = false;
        float fall[2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float top = fmaxf(s[0][2 * r], s[0][2 * r + 1]);
#pragma unroll
          for (int nt = 1; nt < 4; ++nt) top = fmaxf(top, fmaxf(s[nt][2 * r], s[nt][2 * r + 1]));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          // The running "maximum" is what exponents are measured from: the maximum less SHIFT, rounded, and the
          // same number for p, for what is rescaled and for the joins, so that its rounding cancels.
          float mult = S::KV8 ? rs[r] : args.s2;
          if (fabsf(top * mult) >= kFarScore) {
            // Out here a rounded maximum is far from the product that it is rounded from (2^27: 8, which fp16
            // does not stand): scores are rounded first, as coarsely, and the largest has exponent 0.
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) s[nt][2 * r] *= mult, s[nt][2 * r + 1] *= mult;
            top = fmaxf(top * mult, m[r]);
            mult = 1.f;
          } else {
            top = fmaxf(fmaf(top, mult, -S::SHIFT), m[r]);
          }
          const float base = top == -INFINITY ? 0.f : top;
          fall[r] = ex2(m[r] - base);
          grow = grow || top != m[r];
          m[r] = top;
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            // (the exponent is rounded once, near SHIFT where it counts)
            float p0 = ex2(fmaf(s[nt][2 * r], mult, -base)), p1 = ex2(fmaf(s[nt][2 * r + 1], mult, -base));
            sum += p0 + p1;
#pragma unroll
            for (int k = 0; k < S::PT; ++k) pt[r][k][nt] = term<S::KV8>(p0, p1);
          }
          l[r] = l[r] * fall[r] + sum;
        }
        if (__any_sync(~0u, grow)) {
#pragma unroll
          for (int i2 = 0; i2 < D / 8; ++i2) {
            o[i2][0] *= fall[0], o[i2][1] *= fall[0];
            o[i2][2] *= fall[NR - 1], o[i2][3] *= fall[NR - 1];
          }
        }
        // ---- o += p v
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half && !pair) break;
          const int lo = half * 2, hi = half * 2 + 1;
          auto pv = [&](float(&c)[4], uint32_t b0, uint32_t b1) {
            if (S::WIDE) {
#pragma unroll
              for (int k = 0; k < S::PT; ++k) mma(c, pt[0][k][lo], pt[NR - 1][k][lo], pt[0][k][hi], pt[NR - 1][k][hi], b0, b1, S::KV8);
            } else {
              mma(c, pt[0][0][lo], pt[0][1][lo], pt[0][0][hi], pt[0][1][hi], b0, b1, S::KV8);
              if (S::PT > 2) mma(c, 0, pt[0][S::PT - 1][lo], 0, pt[0][S::PT - 1][hi], b0, b1, S::KV8);
            }
          };
          const int slot = half ? stage2 : stage;
          if (!S::KV8) {
            // lanes 0-7, 8-15: rows 0-7 and 8-15 of one chunk, 16-31: of the next
            const int row = lane & 15;
            const uint32_t base = queue + slot * S::STAGE + S::KBYTES + row * D * 2;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              uint32_t b[4];
              asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                           : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                           : "r"(base + (((2 * j + (lane >> 4)) ^ (row & 7)) & (D / 8 - 1)) * 16)
                           : "memory");
              pv(o[2 * j], b[0], b[1]);
              pv(o[2 * j + 1], b[2], b[3]);
            }
          } else {
            const uint8_t* at = queue_at + slot * S::STAGE;
            uint32_t v[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint8_t* p = at + v_slot(r, 0);
              if (S::VB == 16) {
                const uint4 u = *reinterpret_cast<const uint4*>(p);
                v[r][0] = u.x, v[r][1] = u.y, v[r][2] = u.z, v[r][3] = u.w;
              } else {
                const uint2 u = *reinterpret_cast<const uint2*>(p);
                v[r][0] = u.x, v[r][1] = u.y;
              }
            }
#pragma unroll
            for (int i2 = 0; i2 < S::VB / 4; ++i2)
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                // codes of two positions side by side, two dims in a register
                const uint32_t e = __byte_perm(v[0][i2], v[1][i2], h2 ? 0x7362 : 0x5140);
                const uint32_t d = __byte_perm(v[2][i2], v[3][i2], h2 ? 0x7362 : 0x5140);
                pv(o[i2 * 4 + h2 * 2], widen(e), widen(d));
                pv(o[i2 * 4 + h2 * 2 + 1], widen_high(e), widen_high(d));
              }
          }
        }
        bad = bad || (bad_stages >> stage & 1) || (pair && bad_stages >> stage2 & 1);
        __syncwarp();   // all lanes have read what is overwritten
        fetch(stage);
        stage = stage2;
        if (pair) {
          fetch(stage);
          stage = stage + 1 == S::STAGES ? 0 : stage + 1;
        }
      }

      const bool more_of_it = stop > w.i + rank + S::FOLD * team;   // the scratch holds the sum of earlier tiles
#pragma unroll
      for (int r = 0; r < (S::WIDE ? 2 : 1); ++r) {
        const int head = g + 8 * r;
        float* const row = merge + (warp * S::ROWS + head) * D;
        const float back = more_of_it ? ex2(merge_m[warp * S::ROWS + head] - m[r]) : 0.f;
        const auto value = [&](int i2, int half, float before) {
          const float v = S::WIDE ? o[i2][2 * r + half] : o[i2][half] + o[i2][2 + half];
          return more_of_it ? fmaf(before, back, v) : v;
        };
        if (head >= group) continue;
        if (S::KV8) {   // a lane's accumulators are two runs of D / 8 consecutive dims
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i2 = 0; i2 < D / 8; i2 += 4) {
              float4* const p = reinterpret_cast<float4*>(row + S::place(head, (2 * t + half) * (D / 32) + i2 / 4));
              const float4 b = *p;
              *p = make_float4(value(i2, half, b.x), value(i2 + 1, half, b.y), value(i2 + 2, half, b.z), value(i2 + 3, half, b.w));
            }
        } else {
#pragma unroll
          for (int i2 = 0; i2 < D / 8; ++i2) {
            float2* const p = reinterpret_cast<float2*>(row + S::place(head, 2 * i2 + (t >> 1)) + (t & 1) * 2);
            const float2 b = *p;
            *p = make_float2(value(i2, 0, b.x), value(i2, 1, b.y));
          }
        }
      }
      __syncwarp();   // all have read the maximum that the sum was measured from
#pragma unroll
      for (int r = 0; r < (S::WIDE ? 2 : 1); ++r)
        if (t == 0) merge_m[warp * S::ROWS + g + 8 * r] = m[r];
      __syncwarp();
    }

    // ---- the warps' results joined
    const int active = min(w.end - w.i, team);
#pragma unroll
    for (int r = 0; r < (S::WIDE ? 2 : 1); ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
      if (bad) l[r] = __int_as_float(0x7fffffff);
      if (t == 0 && rank < active) merge_l[warp * S::ROWS + g + 8 * r] = l[r];
    }
    worker_sync();
    const bool begins = w.i == 0, ends = w.end == w.s.tiles;
    float* slot = args.parts + (worker * 2ll + begins) * S::SLOT;
    for (int i = (rank * 32 + lane) * 4; i < group * D; i += team * 128) {
      const int head = i / D, d = i % D;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float top = -INFINITY, den = 0.f;
      for (int k = 0; k < active; ++k) top = fmaxf(top, merge_m[(lead + k) * S::ROWS + head]);
      for (int k = 0; k < active; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(merge + ((lead + k) * S::ROWS + head) * D + S::place(head, d / 4));
        const float e = top == -INFINITY ? 0.f : ex2(merge_m[(lead + k) * S::ROWS + head] - top);
        sum.x += e * v.x, sum.y += e * v.y, sum.z += e * v.z, sum.w += e * v.w;
        den += e * merge_l[(lead + k) * S::ROWS + head];
      }
      if (begins && ends) {
        const float f = den == 0 ? 0.f : (S::KV8 ? a.v_scale : 1.f) / den;
        store_out<S::IO32>(a.out_dev, w.b * a.out_seq_stride + (w.h * group + head) * a.out_head_stride + d,
                           make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f));
        if (d == 0 && a.lse_dev)
          a.lse_dev[static_cast<long long>(w.b) * a.n_q_heads + w.h * group + head] = lse_of(top, den);
      } else {
        *reinterpret_cast<float4*>(slot + head * D + d) = sum;
        if (d == 0) slot[S::ROWS * D + head] = top, slot[S::ROWS * (D + 1) + head] = den;
      }
    }
    if (begins && !ends && rank == 0 && lane == 0) {
      args.joins[worker] = make_int4(w.b, w.h, shares.owner(x + w.s.tiles - 1), 0);
    }
    x += w.end - w.i;
    if (w.left == 0) break;
    // All of the worker's warps have read the scratch: one of them may be done with the next segment, and
    // write its maximum and sum there, before a slower one is done with this.
    worker_sync();
    walk_next(a, w);
  }
}

template <class S>
__device__ inline void store_joined(const xlpk_attention_args& a, const int4& j, int head, int d, float4 sum, float top, float den) {
  const float f = den == 0 ? 0.f : (S::KV8 ? a.v_scale : 1.f) / den;
  const int h = j.y * (a.n_q_heads / a.n_kv_heads) + head;
  store_out<S::IO32>(a.out_dev, j.x * a.out_seq_stride + h * a.out_head_stride + d,
                     make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f));
  if (d == 0 && a.lse_dev) a.lse_dev[static_cast<long long>(j.x) * a.n_q_heads + h] = lse_of(top, den);
}

// The pieces of every segment that one worker begins and another ends, joined by their maxima:
// for each query head of the group by one CTA (workers that are CTAs: few segments, up to
// one piece for each SM) or by one warp (many segments of few pieces).
template <class S>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Args args) {
  constexpr int D = S::D, LANES = D / 4, TEAMS = kThreads / LANES;
  __shared__ float4 sums[TEAMS][LANES];
  __shared__ float dens[TEAMS], tops[kJoinWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const xlpk_attention_args& a = args.a;
  const int group = a.n_q_heads / a.n_kv_heads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool by_warp = *args.team == 1;
  const int item = by_warp ? blockIdx.x * kJoinWarps + warp : blockIdx.x, head = item % group, worker = item / group;
  if (worker >= args.ctas * (by_warp ? S::WARPS : 1)) return;
  const int4 j = args.joins[worker];
  if (j.x < 0) return;
  const int n = j.z - worker + 1;
  // piece 0 is the slot of the segment that its worker begins, the others continue theirs
  const auto slot = [&](int k) { return args.parts + ((worker + k) * 2ll + (k == 0)) * S::SLOT; };
  const int size = by_warp ? 32 : kThreads, me = by_warp ? lane : threadIdx.x, teams = size / LANES;
  float top = -INFINITY;
  for (int k = me; k < n; k += size) top = fmaxf(top, slot(k)[S::ROWS * D + head]);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (!by_warp) {
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    for (int k = 0; k < kJoinWarps; ++k) top = fmaxf(top, tops[k]);
  }
  const int d = me % LANES, team = me / LANES;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
#pragma unroll 4
  for (int k = team; k < n; k += teams) {
    const float* p = slot(k);
    const float4 v = *reinterpret_cast<const float4*>(p + head * D + d * 4);
    const float e = top == -INFINITY ? 0.f : ex2(p[S::ROWS * D + head] - top);
    sum.x += e * v.x, sum.y += e * v.y, sum.z += e * v.z, sum.w += e * v.w;
    den += e * p[S::ROWS * (D + 1) + head];
  }
  if (!by_warp) {
    sums[team][d] = sum;
    if (d == 0) dens[team] = den;
    __syncthreads();
    if (team != 0) return;
    for (int k = 1; k < TEAMS; ++k) {
      const float4 v = sums[k][d];
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      den += dens[k];
    }
  } else if (LANES < 32) {
    for (int o = LANES; o < 32; o <<= 1) {
      sum.x += __shfl_xor_sync(~0u, sum.x, o), sum.y += __shfl_xor_sync(~0u, sum.y, o);
      sum.z += __shfl_xor_sync(~0u, sum.z, o), sum.w += __shfl_xor_sync(~0u, sum.w, o);
      den += __shfl_xor_sync(~0u, den, o);
    }
    if (team != 0) return;
  }
  store_joined<S>(a, j, head, d * 4, sum, top, den);
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
  if (a->n_q_heads > 1 << 20)   // (a row of them is counted in 32 bits)
    return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_decode_attention: more than 2^20 query heads");
  if ((a->io_dtype != XLPK_DTYPE_BF16 && a->io_dtype != XLPK_DTYPE_FP32) ||
      (a->kv_dtype != XLPK_DTYPE_BF16 && a->kv_dtype != XLPK_DTYPE_FP8_E4M3))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: io_dtype is bf16 or fp32, kv_dtype bf16 or e4m3");
  if (a->n_pages < 0 || a->page_size < 1 || a->table_cols < 0 || a->window < 0 || a->sinks < 0)
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: a negative count");
  if (static_cast<int64_t>(a->table_cols) * a->page_size > INT32_MAX - 4 * kTile)
    return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_decode_attention: a capacity of 2^31 - 64 positions or more");
  if (!(a->scale > 0) || !(a->scale < 0x1p127f))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: scale is not positive and below 2^127");
  if (a->kv_dtype == XLPK_DTYPE_FP8_E4M3 && (!power_of_two_scale(a->k_scale) || !power_of_two_scale(a->v_scale)))
    return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: cache scales are powers of two in [2^-24, 2^24]");
  if (static_cast<int64_t>(a->n_seqs) * a->n_kv_heads >
      INT32_MAX / (static_cast<int64_t>(a->table_cols) * a->page_size / kTile + 2))
    return refuse(XLPK_ERR_UNSUPPORTED, "xlpk_decode_attention: n_seqs * n_kv_heads * capacity of about 2^35 positions or more");
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
  for (int64_t s : io_strides) ok = ok && s >= 0 && (s * io) % 16 == 0;
  for (int64_t s : kv_strides) ok = ok && s >= 0 && (s * kv) % 16 == 0;
  ok = ok && a->table_stride >= 0;
  if (!ok) return refuse(XLPK_ERR_INVALID_ARG, "xlpk_decode_attention: a pointer or stride is not a multiple of 16 bytes, or negative");
  return XLPK_OK;
}

template <class S>
xlpk_status launch(const Args& args, int ctas, cudaStream_t st) {
  static std::atomic<unsigned long long> ready;   // devices whose kernel has its shared memory
  int dev = 0;
  XLPK_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    XLPK_CUDA(cudaFuncSetAttribute(attention_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM));
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  attention_kernel<S><<<ctas, S::THREADS, S::SMEM, st>>>(args);
  XLPK_CUDA(cudaGetLastError());
  cudaLaunchConfig_t c{};
  const int group = args.a.n_q_heads / args.a.n_kv_heads;
  c.gridDim = dim3(std::max(ctas * group, (ctas * S::WARPS * group + kJoinWarps - 1) / kJoinWarps));
  c.blockDim = dim3(kThreads);
  c.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &early;
  c.numAttrs = 1;
  XLPK_CUDA(cudaLaunchKernelEx(&c, join_kernel<S>, args));
  return XLPK_OK;
}

template <int D, bool KV8>
xlpk_status launch_for(const Args& args, int ctas, cudaStream_t st) {
  const bool io32 = args.a.io_dtype == XLPK_DTYPE_FP32;
  if (args.a.n_q_heads / args.a.n_kv_heads > 8)
    return io32 ? launch<Shape<D, KV8, true, true>>(args, ctas, st) : launch<Shape<D, KV8, true, false>>(args, ctas, st);
  return io32 ? launch<Shape<D, KV8, false, true>>(args, ctas, st) : launch<Shape<D, KV8, false, false>>(args, ctas, st);
}

constexpr int kMaxWorkers = kMaxCtas * 12;
constexpr int64_t kJoinBytes = (kMaxWorkers + 1) * sizeof(int4);

}  // namespace

extern "C" int64_t xlpk_decode_attention_workspace(const xlpk_attention_args* a) {
  if (!shape_ok(a)) return 0;
  // (12 warps of 8 rows at most, or 8 of 16)
  return kJoinBytes + kMaxCtas * 8 * 2 * 16 * (static_cast<int64_t>(a->head_dim) + 2) * 4;
}

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
  Args args;
  args.a = *a;
  // (copies of rows that are not there read nothing, but name the pool's start: with no pages, some memory)
  if (a->n_pages == 0) args.a.k_dev = args.a.v_dev = workspace_dev;
  const double s2 = static_cast<double>(a->scale) * 1.4426950408889634074;
  args.exp = 0;
  args.s2 = static_cast<float>(a->kv_dtype == XLPK_DTYPE_FP8_E4M3 ? std::frexp(s2 * a->k_scale, &args.exp) : s2);
  args.page_shift = (a->page_size & (a->page_size - 1)) == 0 ? __builtin_ctz(a->page_size) : -1;
  args.flat = a->page_size % kTile == 0 || a->table_cols == 1;   // (behind its only page no position is visible)
  args.ctas = std::min(sms, kMaxCtas);
  args.joins = static_cast<int4*>(workspace_dev);
  args.team = reinterpret_cast<int*>(args.joins + kMaxWorkers);
  args.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace_dev) + kJoinBytes);
  const int ctas = args.ctas;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->head_dim == 64)
    return a->kv_dtype == XLPK_DTYPE_BF16 ? launch_for<64, false>(args, ctas, st) : launch_for<64, true>(args, ctas, st);
  return a->kv_dtype == XLPK_DTYPE_BF16 ? launch_for<128, false>(args, ctas, st) : launch_for<128, true>(args, ctas, st);
}
