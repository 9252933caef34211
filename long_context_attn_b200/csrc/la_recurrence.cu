// Gated linear recurrence h_t = a_t h_{t-1} + b_t, a = sigmoid(f), b = x or (1 - a) x, channel
// by channel: forward, one-token step and backward (sm_100a).
//
// Rows t .. u of a channel act on the state that enters them as h -> A h + H, A the product of
// their gates; two neighbours compose to (A2 A1, A2 H1 + H2).  The packed rows are cut into
// tiles of L rows x C channels, one CTA each, and a tile is read once: every thread folds its R
// rows x V channels in registers, the CTA folds the threads, the tile's (A, H) is published,
// the state entering the tile is found from the tiles before it, and the threads walk their rows
// again from the states that enter them.  A row that starts a sequence takes its state from
// state_in instead, so packed sequences need no tiles of their own and cut the dependence.
//
// State entering a tile: tiles are handed out in time order by a ticket, so every tile before
// one that is worked on has been started and never waits for a later one.  A warp looks back over
// the tiles before its own until it finds one whose state after the last row is known, and folds
// the (A, H) between from there, oldest first.  Values and their being there are one word, read
// and written whole, so the chain needs no flags and no fences.  That fold does the same operations in the same
// order as the tiles' own (h <- A h + H, tile by tile), so the result does not depend on how
// far the warp had to look.
//
// The backward walks time in reverse: with c_t = a_t (dout_t + c_{t+1}) what flows into the
// state before row t, rows act on the c that enters them from behind as c -> A c + C with the same
// A.  h is recomputed from the checkpoint that the tile's first row starts from.
#include "la_common.cuh"

namespace la {

void set_last_path(const char* path);

namespace {

constexpr int kCkRows = LA_RECURRENCE_CHECKPOINT_ROWS;
constexpr int kThreads = 256;
#ifndef FB
#define FB 2
#endif
#ifndef BB
#define BB 2
#endif
#ifndef FSV
#define FSV 8
#define FSC 8
#define FSR 4
#endif
#ifndef BSV
#define BSV 4
#define BSC 8
#define BSR 4
#endif

struct RecArgs {
  const void *x, *f, *dout;
  void *out, *dx, *df;
  const float *s0, *ds1;
  float *s1, *ds0, *ck;
  const int* cu;
  int nseq, T, W, tied;
  int64_t tokens;
  ErrRec* err;
  // Chain between the tiles (more than one in time): all bits set before each walk.
  int ntiles, nblocks;          // in time, across the channels
  unsigned int* ticket;         // [0]: the last tile handed out; [1]: kOpen, until a wait ran out
  uint64_t* agg;                // [ntiles][nblocks * C]: (A, H) of the tile
  unsigned int* inc;            // [ntiles][nblocks * C]: state after the tile
};
// What a word of the chain holds until its value is there: a NaN that is never published.
constexpr unsigned int kOpen = 0xFFFFFFFFu;

// Two fp32 operations in one instruction (each rounded as the single one).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
      " fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a; }"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// a = sigmoid(f) = 1 / (1 + t) and keep = 1 - a = t / (1 + t) with t = exp(-f), neither by
// cancellation.  Two special-function operations an element, exp2 and the reciprocal, which the
// memory rate leaves room for.  bf16 gates take exp2 of the rounded product -f log2(e): t is
// then off by at most (4 + |f|) 2^-24, against the 2^-9 the gate itself is rounded to (with expf
// and an IEEE division the first tiled kernel spent 47 instructions an element and ran at 0.30
// of the HBM rate, instruction-bound); fp32 gates call expf.  a is 0 where t leaves fp32's
// normal range (f < -87.3), and keep, which t a would not give there, is 1.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename T> __device__ __forceinline__ void gates(float2 f, float2& a, float2& keep) {
  float2 t;
  if constexpr (sizeof(T) == 2) {
    const float2 y = mul2(f, splat(-1.4426950408889634f));
    t = make_float2(exp2_approx(y.x), exp2_approx(y.y));
  } else {
    t = make_float2(expf(-f.x), expf(-f.y));
  }
  const float2 d = add2(t, splat(1.0f));
  a = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  const float2 k = mul2(t, a);
  keep = make_float2(a.x == 0.0f ? 1.0f : k.x, a.y == 0.0f ? 1.0f : k.y);
}

// V consecutive channels of one row, as loaded; they are worked on in pairs (V = 1: with an idle
// second half).
template <typename T, int V> struct Pack;
template <> struct Pack<uint16_t, 8> {
  uint4 r;
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ __forceinline__ static Pack from(const float2* o) {
    return Pack{make_uint4(pack_bf16x2(o[0].x, o[0].y), pack_bf16x2(o[1].x, o[1].y), pack_bf16x2(o[2].x, o[2].y),
                           pack_bf16x2(o[3].x, o[3].y))};
  }
};
template <> struct Pack<uint16_t, 4> {
  uint2 r;
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t w = i == 0 ? r.x : r.y;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ __forceinline__ static Pack from(const float2* o) {
    return Pack{make_uint2(pack_bf16x2(o[0].x, o[0].y), pack_bf16x2(o[1].x, o[1].y))};
  }
};
template <> struct Pack<float, 4> {
  float4 r;
  __device__ __forceinline__ float2 pair(int i) const { return i == 0 ? make_float2(r.x, r.y) : make_float2(r.z, r.w); }
  __device__ __forceinline__ static Pack from(const float2* o) { return Pack{make_float4(o[0].x, o[0].y, o[1].x, o[1].y)}; }
};
template <> struct Pack<uint16_t, 1> {
  uint16_t r;
  __device__ __forceinline__ float2 pair(int) const { return make_float2(bf16_bits_to_f32(r), 0.f); }
  __device__ __forceinline__ static Pack from(const float2* o) { return Pack{f32_to_bf16_bits(o[0].x)}; }
};
template <> struct Pack<float, 1> {
  float r;
  __device__ __forceinline__ float2 pair(int) const { return make_float2(r, 0.f); }
  __device__ __forceinline__ static Pack from(const float2* o) { return Pack{o[0].x}; }
};
// V fp32 values of the states, the checkpoints or the folds.
template <int V> __device__ __forceinline__ void load_f32(const float* p, float2* o) {
  if constexpr (V == 1) {
    o[0] = make_float2(*p, 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 t = *reinterpret_cast<const float4*>(p + i);
      o[i / 2] = make_float2(t.x, t.y);
      o[i / 2 + 1] = make_float2(t.z, t.w);
    }
  }
}
template <int V> __device__ __forceinline__ void store_f32(float* p, const float2* o) {
  if constexpr (V == 1) {
    *p = o[0].x;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(o[i / 2].x, o[i / 2].y, o[i / 2 + 1].x, o[i / 2 + 1].y);
  }
}

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// CL threads side by side take V channels each; G = 256 / CL groups of them take R rows each.
template <typename T_, int V_, int CL_, int R_> struct Shape {
  using T = T_;
  static constexpr int V = V_, CL = CL_, R = R_, U = (V + 1) / 2;   // U pairs
  static constexpr int C = CL * V, G = kThreads / CL, L = G * R;
  static constexpr int NP = kThreads / C, GP = G / NP;   // the fold over groups: NP threads a channel
  static_assert(C % 32 == 0 && kThreads % C == 0 && G % NP == 0 && L == kCkRows, "tile");
};

// A tile: its place in the walk and across the channels, whether a sequence starts or ends in its
// rows (or they end), and the sequence of its first row (the first that ends behind it).
struct Tile {
  int k, cb, any, seq;
};

template <class S, int NT, int NB> struct Smem {
  Pack<typename S::T, S::V> raw[NB][NT][S::R][kThreads];   // each thread's own, as the copies bring them
  float A[S::G][S::C], H[S::G][S::C];     // of each group; then H: the state entering it
  float pA[S::NP][S::C], pH[S::NP][S::C];
  float in[S::C];
  int start[2][S::L], end[2][S::L];       // of a tile with `any`: the sequence that starts (ends) at a row, or -1
  int reset[S::G], preset[S::NP];
  Tile tile[3];
};
// The backward's: the same for the walk back (C, cin, creset) beside the walk forward in the tile.
template <class S, int NT, int NB> struct SmemBack : Smem<S, NT, NB> {
  float Cc[S::G][S::C], pC[S::NP][S::C], cin[S::C];
  int creset[S::G], cpreset[S::NP];
};

// One vector into shared memory without waiting for it; zeros where `in` is false.
template <typename P> __device__ __forceinline__ void copy_async(P* dst, const void* src, bool in) {
  const unsigned int d = static_cast<unsigned int>(__cvta_generic_to_shared(dst));
  if constexpr (sizeof(P) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(in ? 16 : 0) : "memory");
  else if constexpr (sizeof(P) == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(in ? 8 : 0) : "memory");
  else
    *dst = in ? *static_cast<const P*>(src) : P{};   // single elements: waited for
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ unsigned int load_relaxed(const unsigned int* p) {
  unsigned int v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t load_relaxed(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_relaxed(unsigned int* p, unsigned int v) {
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void store_relaxed(uint64_t* p, uint64_t v) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
// The bits of a value of the chain: any NaN as the one that is not kOpen.
__device__ __forceinline__ unsigned int published(float v) { return v == v ? __float_as_uint(v) : 0x7FC00000u; }

// Rows of the packed batch that belong to a sequence: the first `limit` ones.
__device__ __forceinline__ int64_t row_limit(const RecArgs& p) {
  if (!p.cu) return p.tokens;
  const int64_t n = __ldg(p.cu + p.nseq);
  return n < 0 ? 0 : n < p.tokens ? n : p.tokens;
}

// Completes a tile (one thread).  Without `any`, every row of the tile is in one sequence and none
// is its first or last.
template <class S> __device__ __forceinline__ void look_up(const RecArgs& p, int64_t r0, int64_t limit, Tile& t) {
  constexpr int L = S::L;
  if (!p.cu) {
    const unsigned int T = p.T, row = static_cast<unsigned int>(r0), s = row / T, in = row - s * T;
    t.seq = static_cast<int>(s);
    t.any = in == 0 || static_cast<int64_t>(in) + L >= T || r0 + L > limit;
    return;
  }
  int lo = 0, hi = p.nseq;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid + 1) > r0) hi = mid; else lo = mid + 1;
  }
  t.seq = lo;
  t.any = lo >= p.nseq || __ldg(p.cu + lo) >= r0 || __ldg(p.cu + lo + 1) <= r0 + L || r0 + L > limit;
}

// Marks the rows of a tile with `any` where sequences start and end (a thread a row).
template <class S>
__device__ __forceinline__ void mark_rows(const RecArgs& p, int64_t r0, int64_t limit, int seq, int* start, int* end) {
  const int tid = threadIdx.x;
  if (tid >= S::L) return;
  const int64_t row = r0 + tid;
  int st = -1, en = -1;
  if (row < limit) {
    if (!p.cu) {
      const unsigned int T = p.T, s = static_cast<unsigned int>(row) / T, in = static_cast<unsigned int>(row) - s * T;
      if (in == 0) st = static_cast<int>(s);
      if (in == T - 1) en = static_cast<int>(s);
    } else {
      int a = seq, b = p.nseq;   // the sequence of this row
      while (a < b) {
        const int mid = (a + b) >> 1;
        if (__ldg(p.cu + mid + 1) > row) b = mid; else a = mid + 1;
      }
      if (a < p.nseq) {
        const int64_t first = __ldg(p.cu + a), last = static_cast<int64_t>(__ldg(p.cu + a + 1)) - 1;
        if (first >= 0 && first <= row && last < p.tokens) {
          if (first == row) st = a;
          if (last == row) en = a;
        }
      }
    }
  }
  start[tid] = st;
  end[tid] = en;
}

// Sequences without rows: their final state (gradient) is the initial (final) one.  Malformed
// offsets are reported.  A warp a sequence.
__device__ __forceinline__ void rowless_sequences(const RecArgs& p, const float* from, float* to) {
  if (!p.cu) return;
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kThreads / 32);
  for (int64_t s = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); s < p.nseq; s += warps) {
    const int a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1);
    if (a < 0 || b < a || b > p.tokens || (s == 0 && a != 0)) {
      if (lane == 0) report(p.err, LA_ERR_DEVICE, SITE_VARLEN_CU, static_cast<unsigned>(s), 0);
    } else if (a == b && to) {
      for (int c = lane; c < p.W; c += 32) to[s * p.W + c] = from ? from[s * p.W + c] : 0.f;
    }
  }
}

// One warp, 32 channels, `col` the lane's: what enters the walk's tile k (> 0).
__device__ __forceinline__ float look_back(const RecArgs& p, int k, int64_t col, int64_t cols) {
  constexpr int K = 8;   // tiles looked at in one trip to L2
  uint64_t t0 = 0;
  int base = k - 1;
  float h = 0.f;
  for (unsigned int polls = 0;;) {
    unsigned int inc[K], known = 0, there = 0;
    uint64_t agg[K];
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const int i = base - u < 0 ? 0 : base - u;
      inc[u] = load_relaxed(p.inc + i * cols + col);
      agg[u] = load_relaxed(p.agg + i * cols + col);
    }
#pragma unroll
    for (int u = 0; u < K; ++u) {
      known |= static_cast<unsigned int>(inc[u] != kOpen) << u;
      there |= static_cast<unsigned int>(static_cast<unsigned int>(agg[u]) != kOpen) << u;
    }
    known = __reduce_and_sync(0xffffffffu, known);
    there = __reduce_and_sync(0xffffffffu, there);
    const unsigned int near = known ? (known & (0u - known)) - 1u : (1u << K) - 1u;   // tiles nearer than a known one
    if ((there & near) == near) {
      if (!known) {
        base -= K;   // all (A, H) there: look further back
        continue;
      }
      // the known state, then the tiles of this window behind it, oldest first
#pragma unroll
      for (int u = K - 1; u >= 0; --u) {
        if (near >> u & 1u)
          h = fmaf(__uint_as_float(static_cast<unsigned int>(agg[u])), h,
                   __uint_as_float(static_cast<unsigned int>(agg[u] >> 32)));
        else if (known >> u & 1u)
          h = __uint_as_float(inc[u]);
      }
      break;
    }
    if ((++polls & 63u) == 0) {   // no progress: has somebody given up, or is it time to?
      if (load_relaxed(p.ticket + 1) != kOpen) return 0.f;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > wait_limit_ns(p.err)) {
        if ((threadIdx.x & 31) == 0) {
          report(p.err, LA_ERR_TIMEOUT, SITE_RECURRENCE_CHAIN, static_cast<unsigned>(k), static_cast<unsigned>(col));
          store_relaxed(p.ticket + 1, 0u);
        }
        return 0.f;
      }
    }
  }
  for (int i = base + 1; i < k; i += K) {   // the windows passed on the way
    uint64_t t[K];
#pragma unroll
    for (int u = 0; u < K; ++u) t[u] = load_relaxed(p.agg + (i + u) * cols + col);
#pragma unroll
    for (int u = 0; u < K; ++u)
      h = fmaf(__uint_as_float(static_cast<unsigned int>(t[u])), h, __uint_as_float(static_cast<unsigned int>(t[u] >> 32)));
  }
  return h;
}

// What the chain knows of the walk's tile k is (tA, tH), with `cut` set where a sequence starts
// in it, so that what enters it does not leave it: published; returns what enters the tile.
// `meanwhile` runs before the wait.  One warp, 32 channels, `col` the lane's.
template <class F>
__device__ __forceinline__ float chain(const RecArgs& p, int k, int64_t col, int64_t cols, float tA, float tH, int cut,
                                       F meanwhile) {
  if (p.ntiles == 1) {
    meanwhile();
    return 0.f;
  }
  if (cut || k == 0)
    store_relaxed(p.inc + k * cols + col, published(tH));
  else
    store_relaxed(p.agg + k * cols + col, static_cast<uint64_t>(published(tH)) << 32 | published(tA));
  meanwhile();
  if (k == 0) return 0.f;   // nothing enters the first tile
  const float in = look_back(p, k, col, cols);
  if (!cut) store_relaxed(p.inc + k * cols + col, published(fmaf(tA, in, tH)));
  return in;
}

// Acts on h as a run of rows with (A, H) does; `cut`: what enters the run does not leave it (and
// is not multiplied by 0: it may be infinite).
__device__ __forceinline__ float act(int cut, float A, float H, float h) { return cut ? H : fmaf(A, h, H); }

// The fold over the CTA's groups and, through the chain, over the tiles before it.  On entry sm.A,
// sm.H, sm.reset hold each group's (A, H) and whether a sequence starts in it; on return sm.H[g]
// is what enters group g.  `meanwhile` runs once in every thread, before the wait.
template <class S, class M, class F>
__device__ __forceinline__ void fold_forward(const RecArgs& p, M& sm, int k, int cb, F meanwhile) {
  constexpr int C = S::C, NP = S::NP, GP = S::GP;
  const int c = threadIdx.x % C, part = threadIdx.x / C;
  float A[GP], H[GP];
  float pa = 1.f, ph = 0.f;
  int pr = 0;
#pragma unroll
  for (int i = 0; i < GP; ++i) {
    const int g = part * GP + i, r = sm.reset[g];
    A[i] = sm.A[g][c];
    H[i] = sm.H[g][c];
    ph = act(r, A[i], H[i], ph);
    pa *= A[i];
    pr |= r;
  }
  sm.pA[part][c] = pa;
  sm.pH[part][c] = ph;
  if (c == 0) sm.preset[part] = pr;
  __syncthreads();
  if (part == 0) {   // whole warps: C is a multiple of 32
    float tA = 1.f, tH = 0.f;
    int cut = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      tH = act(sm.preset[i], sm.pA[i][c], sm.pH[i][c], tH);
      tA *= sm.pA[i][c];
      cut |= sm.preset[i];
    }
    sm.in[c] = chain(p, k, static_cast<int64_t>(cb) * C + c, static_cast<int64_t>(p.nblocks) * C, tA, tH, cut, meanwhile);
  } else {
    meanwhile();
  }
  __syncthreads();
  float h = sm.in[c];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (i < part) h = act(sm.preset[i], sm.pA[i][c], sm.pH[i][c], h);
#pragma unroll
  for (int i = 0; i < GP; ++i) {
    const int g = part * GP + i;
    sm.H[g][c] = h;
    h = act(sm.reset[g], A[i], H[i], h);
  }
  __syncthreads();
}

// The backward's folds, both at once: forward in the tile from the checkpoint `ck` (the thread's
// channel's), and from the last group to the first, through the chain, of what flows back:
// on return sm.H[g] and sm.Cc[g] are what enters group g from before and from behind.
template <class S, class M, class F>
__device__ __forceinline__ void fold_both(const RecArgs& p, M& sm, int k, int cb, float ck, F meanwhile) {
  constexpr int C = S::C, NP = S::NP, GP = S::GP;
  const int c = threadIdx.x % C, part = threadIdx.x / C;
  float A[GP], H[GP], Cc[GP];
  float pa = 1.f, ph = 0.f, pc = 0.f;
  int pr = 0, pe = 0;
#pragma unroll
  for (int i = 0; i < GP; ++i) {
    const int g = part * GP + i, r = sm.reset[g];
    A[i] = sm.A[g][c];
    H[i] = sm.H[g][c];
    Cc[i] = sm.Cc[g][c];
    ph = act(r, A[i], H[i], ph);
    pa *= A[i];
    pr |= r;
  }
#pragma unroll
  for (int i = GP - 1; i >= 0; --i) {
    const int e = sm.creset[part * GP + i];
    pc = act(e, A[i], Cc[i], pc);
    pe |= e;
  }
  sm.pA[part][c] = pa;
  sm.pH[part][c] = ph;
  sm.pC[part][c] = pc;
  if (c == 0) {
    sm.preset[part] = pr;
    sm.cpreset[part] = pe;
  }
  __syncthreads();
  if (part == 0) {
    float tA = 1.f, tC = 0.f;
    int cut = 0;
#pragma unroll
    for (int i = NP - 1; i >= 0; --i) {
      tC = act(sm.cpreset[i], sm.pA[i][c], sm.pC[i][c], tC);
      tA *= sm.pA[i][c];
      cut |= sm.cpreset[i];
    }
    sm.cin[c] = chain(p, k, static_cast<int64_t>(cb) * C + c, static_cast<int64_t>(p.nblocks) * C, tA, tC, cut, meanwhile);
  } else {
    meanwhile();
  }
  float h = ck;
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (i < part) h = act(sm.preset[i], sm.pA[i][c], sm.pH[i][c], h);
#pragma unroll
  for (int i = 0; i < GP; ++i) {
    const int g = part * GP + i;
    sm.H[g][c] = h;
    h = act(sm.reset[g], A[i], H[i], h);
  }
  __syncthreads();
  float b = sm.cin[c];
#pragma unroll
  for (int i = NP - 1; i >= 0; --i)
    if (i > part) b = act(sm.cpreset[i], sm.pA[i][c], sm.pC[i][c], b);
#pragma unroll
  for (int i = GP - 1; i >= 0; --i) {
    const int g = part * GP + i;
    sm.Cc[g][c] = b;
    b = act(sm.creset[g], A[i], Cc[i], b);
  }
  __syncthreads();
}

// The tiles a CTA works on, one after the other: by ticket where tiles wait for one another, so
// that a tile is only waited for once somebody works on it (tickets are drawn ahead, but in
// order: the holder of the smallest unfinished one works on it), else dealt out.
__device__ __forceinline__ int next_tile(const RecArgs& p, int nth) {
  if (p.ntiles > 1) return static_cast<int>(atomicAdd(p.ticket, 1u) + 1u);
  return static_cast<int>(blockIdx.x + static_cast<unsigned int>(nth) * gridDim.x);
}
__device__ __forceinline__ void place(const RecArgs& p, int tile, Tile& t) {
  t.k = tile / p.nblocks;
  t.cb = tile - t.k * p.nblocks;
}

// Both walks.  Ahead of the tile being worked on, the next one's rows are on their way into shared
// memory and the one's after it are asked for; `scout`, a thread of the last warp, draws and looks
// up the tiles while the first warps wait for the chain.
template <class S, bool TIED> __global__ void __launch_bounds__(kThreads, FB) rec_forward_kernel(RecArgs p) {
  using T = typename S::T;
  using P = Pack<T, S::V>;
  constexpr int V = S::V, R = S::R, U = S::U;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<Smem<S, 2, 2>*>(smem_raw);
  const int tid = threadIdx.x, cl = tid % S::CL, g = tid / S::CL;
  const bool scout = tid == kThreads - 32;
  const int64_t limit = row_limit(p);
  const int filled = static_cast<int>((limit + S::L - 1) / S::L);   // tiles with rows, in time
  rowless_sequences(p, p.s0, p.s1);

  auto fetch = [&](const Tile& t, int buf) {   // a group for every call, so that they can be counted
    if (t.k < filled) {
      const int64_t row0 = static_cast<int64_t>(t.k) * S::L + g * R;
      const int c0 = t.cb * S::C + cl * V;
      const T* x = static_cast<const T*>(p.x) + row0 * p.W + c0;
      const T* f = static_cast<const T*>(p.f) + row0 * p.W + c0;
      if (c0 < p.W && row0 + R <= limit) {
#pragma unroll
        for (int i = 0; i < R; ++i, x += p.W, f += p.W) {
          copy_async(&sm.raw[buf][0][i][tid], x, true);
          copy_async(&sm.raw[buf][1][i][tid], f, true);
        }
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i, x += p.W, f += p.W) {
          const bool in = c0 < p.W && row0 + i < limit;
          copy_async(&sm.raw[buf][0][i][tid], in ? x : static_cast<const T*>(p.x), in);
          copy_async(&sm.raw[buf][1][i][tid], in ? f : static_cast<const T*>(p.f), in);
        }
      }
    }
    copy_commit();
  };
  if (scout) {
    for (int n = 0; n < 2; ++n) {
      place(p, next_tile(p, n), sm.tile[n]);
      if (sm.tile[n].k < filled) look_up<S>(p, static_cast<int64_t>(sm.tile[n].k) * S::L, limit, sm.tile[n]);
    }
  }
  __syncthreads();
  Tile tile = sm.tile[0];
  fetch(tile, 0);
  fetch(sm.tile[1], 1);
  if (tile.k < filled && tile.any)
    mark_rows<S>(p, static_cast<int64_t>(tile.k) * S::L, limit, tile.seq, sm.start[0], sm.end[0]);
  __syncthreads();
  int slot = 0;   // n % 3
  for (int n = 0; tile.k < filled; ++n) {
    const int buf = n & 1, slot1 = slot == 2 ? 0 : slot + 1, slot2 = slot1 == 2 ? 0 : slot1 + 1;
    const int64_t row0 = static_cast<int64_t>(tile.k) * S::L + g * R;
    const int c0 = tile.cb * S::C + cl * V;
    const bool in = c0 < p.W;
    int drawn = 0;
    if (scout) drawn = next_tile(p, n + 2);
    copy_wait<1>();

    float2 a[R][U], b[R][U], A[U], H[U];
    int reset = 0;
#pragma unroll
    for (int e = 0; e < U; ++e) { A[e] = splat(1.f); H[e] = splat(0.f); }
    auto rows_in = [&](auto marked) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const P xr = sm.raw[buf][0][i][tid], fr = sm.raw[buf][1][i][tid];
        if constexpr (decltype(marked)::value) {
          const int s = sm.start[buf][g * R + i];
          if (s >= 0) {
            reset = 1;
#pragma unroll
            for (int e = 0; e < U; ++e) H[e] = splat(0.f);
            if (p.s0 && in) load_f32<V>(p.s0 + static_cast<int64_t>(s) * p.W + c0, H);
          }
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
          float2 keep;
          gates<T>(fr.pair(e), a[i][e], keep);
          b[i][e] = TIED ? mul2(keep, xr.pair(e)) : xr.pair(e);
          H[e] = fma2(a[i][e], H[e], b[i][e]);
          A[e] = mul2(A[e], a[i][e]);
        }
      }
    };
    if (tile.any) rows_in(Yes{}); else rows_in(No{});
    store_f32<V>(&sm.A[g][cl * V], A);
    store_f32<V>(&sm.H[g][cl * V], H);
    if (cl == 0) sm.reset[g] = reset;
    if (scout) place(p, drawn, sm.tile[slot2]);
    __syncthreads();
    const Tile next = sm.tile[slot1];
    fold_forward<S>(p, sm, tile.k, tile.cb, [&] {
      fetch(sm.tile[slot2], buf);
      if (next.k < filled && next.any)
        mark_rows<S>(p, static_cast<int64_t>(next.k) * S::L, limit, next.seq, sm.start[buf ^ 1], sm.end[buf ^ 1]);
      if (scout && sm.tile[slot2].k < filled)
        look_up<S>(p, static_cast<int64_t>(sm.tile[slot2].k) * S::L, limit, sm.tile[slot2]);
    });

    if (in) {
      float2 h[U];
      load_f32<V>(&sm.H[g][cl * V], h);
      T* out = p.out ? static_cast<T*>(p.out) + row0 * p.W + c0 : nullptr;
      auto rows_out = [&](auto marked) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if constexpr (decltype(marked)::value) {
            if (row0 + i >= limit) break;
            const int s = sm.start[buf][g * R + i];
            if (s >= 0) {
#pragma unroll
              for (int e = 0; e < U; ++e) h[e] = splat(0.f);
              if (p.s0) load_f32<V>(p.s0 + static_cast<int64_t>(s) * p.W + c0, h);
            }
          }
          if (i == 0 && g == 0 && p.ck) store_f32<V>(p.ck + static_cast<int64_t>(tile.k) * p.W + c0, h);
#pragma unroll
          for (int e = 0; e < U; ++e) h[e] = fma2(a[i][e], h[e], b[i][e]);
          if (out) {
            *reinterpret_cast<P*>(out) = P::from(h);
            out += p.W;
          }
          if constexpr (decltype(marked)::value) {
            const int s = sm.end[buf][g * R + i];
            if (s >= 0 && p.s1) store_f32<V>(p.s1 + static_cast<int64_t>(s) * p.W + c0, h);
          }
        }
      };
      if (tile.any) rows_out(Yes{}); else rows_out(No{});
    }
    tile = next;
    slot = slot1;
  }
  copy_wait<0>();
}

template <class S, bool TIED> __global__ void __launch_bounds__(kThreads, BB) rec_backward_kernel(RecArgs p) {
  using T = typename S::T;
  using P = Pack<T, S::V>;
  constexpr int V = S::V, R = S::R, U = S::U;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<SmemBack<S, 3, 2>*>(smem_raw);
  const int tid = threadIdx.x, cl = tid % S::CL, g = tid / S::CL;
  const bool scout = tid == kThreads - 32;
  const int64_t limit = row_limit(p);
  const int filled = static_cast<int>((limit + S::L - 1) / S::L);
  rowless_sequences(p, p.ds1, p.ds0);

  auto first_row = [&](const Tile& t) { return static_cast<int64_t>(filled - 1 - t.k) * S::L; };   // back in time
  auto fetch = [&](const Tile& t, int buf) {
    if (t.k < filled) {
      const int64_t row0 = first_row(t) + g * R;
      const int c0 = t.cb * S::C + cl * V;
      const T* src[3] = {static_cast<const T*>(p.x), static_cast<const T*>(p.f), static_cast<const T*>(p.dout)};
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const T* at = src[q] + row0 * p.W + c0;
#pragma unroll
        for (int i = 0; i < R; ++i, at += p.W) {
          const bool in = c0 < p.W && row0 + i < limit;
          copy_async(&sm.raw[buf][q][i][tid], in ? at : src[q], in);
        }
      }
    }
    copy_commit();
  };
  if (scout) {
    for (int n = 0; n < 2; ++n) {
      place(p, next_tile(p, n), sm.tile[n]);
      if (sm.tile[n].k < filled) look_up<S>(p, first_row(sm.tile[n]), limit, sm.tile[n]);
    }
  }
  __syncthreads();
  Tile tile = sm.tile[0];
  fetch(tile, 0);
  fetch(sm.tile[1], 1);
  if (tile.k < filled && tile.any) mark_rows<S>(p, first_row(tile), limit, tile.seq, sm.start[0], sm.end[0]);
  __syncthreads();
  int slot = 0;   // n % 3
  for (int n = 0; tile.k < filled; ++n) {
    const int buf = n & 1, slot1 = slot == 2 ? 0 : slot + 1, slot2 = slot1 == 2 ? 0 : slot1 + 1;
    const int64_t row0 = first_row(tile) + g * R;
    const int c0 = tile.cb * S::C + cl * V;
    const bool in = c0 < p.W;
    int drawn = 0;
    if (scout) drawn = next_tile(p, n + 2);
    const int cf = tile.cb * S::C + tid % S::C;   // the thread's channel in the fold
    const float ck = cf < p.W ? p.ck[static_cast<int64_t>(filled - 1 - tile.k) * p.W + cf] : 0.f;
    copy_wait<1>();

    // What the rows do to h, forward, and to the flow into the state before them, backward.
    float2 a[R][U], A[U], H[U], cc[U];
    int reset = 0, creset = 0;
#pragma unroll
    for (int e = 0; e < U; ++e) { A[e] = splat(1.f); H[e] = cc[e] = splat(0.f); }
    auto rows_in = [&](auto marked) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const P xr = sm.raw[buf][0][i][tid], fr = sm.raw[buf][1][i][tid];
        if constexpr (decltype(marked)::value) {
          const int s = sm.start[buf][g * R + i];
          if (s >= 0) {
            reset = 1;
#pragma unroll
            for (int e = 0; e < U; ++e) H[e] = splat(0.f);
            if (p.s0 && in) load_f32<V>(p.s0 + static_cast<int64_t>(s) * p.W + c0, H);
          }
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
          float2 keep;
          gates<T>(fr.pair(e), a[i][e], keep);
          H[e] = fma2(a[i][e], H[e], TIED ? mul2(keep, xr.pair(e)) : xr.pair(e));
          A[e] = mul2(A[e], a[i][e]);
        }
      }
#pragma unroll
      for (int i = R - 1; i >= 0; --i) {
        const P dr = sm.raw[buf][2][i][tid];
        if constexpr (decltype(marked)::value) {
          const int s = sm.end[buf][g * R + i];
          if (s >= 0) {
            creset = 1;
#pragma unroll
            for (int e = 0; e < U; ++e) cc[e] = splat(0.f);
            if (p.ds1 && in) load_f32<V>(p.ds1 + static_cast<int64_t>(s) * p.W + c0, cc);
          }
        }
#pragma unroll
        for (int e = 0; e < U; ++e) cc[e] = mul2(a[i][e], add2(dr.pair(e), cc[e]));
      }
    };
    if (tile.any) rows_in(Yes{}); else rows_in(No{});
    store_f32<V>(&sm.A[g][cl * V], A);
    store_f32<V>(&sm.H[g][cl * V], H);
    store_f32<V>(&sm.Cc[g][cl * V], cc);
    if (cl == 0) {
      sm.reset[g] = reset;
      sm.creset[g] = creset;
    }
    if (scout) place(p, drawn, sm.tile[slot2]);
    __syncthreads();
    const Tile next = sm.tile[slot1];
    fold_both<S>(p, sm, tile.k, tile.cb, ck, [&] {
      if (next.k < filled && next.any)
        mark_rows<S>(p, first_row(next), limit, next.seq, sm.start[buf ^ 1], sm.end[buf ^ 1]);
      if (scout && sm.tile[slot2].k < filled) look_up<S>(p, first_row(sm.tile[slot2]), limit, sm.tile[slot2]);
    });

    if (in) {
      float2 prev[R][U], h[U];
      load_f32<V>(&sm.H[g][cl * V], h);
      load_f32<V>(&sm.Cc[g][cl * V], cc);
      const int64_t last = (row0 + R - 1) * p.W + c0;
      T* dx = static_cast<T*>(p.dx) + last;
      T* df = static_cast<T*>(p.df) + last;
      auto rows_out = [&](auto marked) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if constexpr (decltype(marked)::value) {
            const int s = sm.start[buf][g * R + i];
            if (s >= 0) {
#pragma unroll
              for (int e = 0; e < U; ++e) h[e] = splat(0.f);
              if (p.s0) load_f32<V>(p.s0 + static_cast<int64_t>(s) * p.W + c0, h);
            }
          }
          const P xr = sm.raw[buf][0][i][tid], fr = sm.raw[buf][1][i][tid];
#pragma unroll
          for (int e = 0; e < U; ++e) {
            prev[i][e] = h[e];
            if (i + 1 < R) {
              float2 again, keep;
              if (TIED) gates<T>(fr.pair(e), again, keep);
              h[e] = fma2(a[i][e], h[e], TIED ? mul2(keep, xr.pair(e)) : xr.pair(e));
            }
          }
        }
#pragma unroll
        for (int i = R - 1; i >= 0; --i, dx -= p.W, df -= p.W) {
          if constexpr (decltype(marked)::value) {
            if (row0 + i >= limit) continue;
            const int s = sm.end[buf][g * R + i];
            if (s >= 0) {
#pragma unroll
              for (int e = 0; e < U; ++e) cc[e] = splat(0.f);
              if (p.ds1) load_f32<V>(p.ds1 + static_cast<int64_t>(s) * p.W + c0, cc);
            }
          }
          const P xr = sm.raw[buf][0][i][tid], fr = sm.raw[buf][1][i][tid], dr = sm.raw[buf][2][i][tid];
          float2 ox[U], of[U];
#pragma unroll
          for (int e = 0; e < U; ++e) {
            float2 again, keep;
            gates<T>(fr.pair(e), again, keep);
            const float2 G1 = add2(dr.pair(e), cc[e]);
            ox[e] = TIED ? mul2(keep, G1) : G1;
            cc[e] = mul2(a[i][e], G1);
            const float2 d = TIED ? fma2(xr.pair(e), splat(-1.f), prev[i][e]) : prev[i][e];
            of[e] = mul2(mul2(keep, cc[e]), d);
          }
          *reinterpret_cast<P*>(dx) = P::from(ox);
          *reinterpret_cast<P*>(df) = P::from(of);
          if constexpr (decltype(marked)::value) {
            const int s = sm.start[buf][g * R + i];
            if (s >= 0 && p.ds0) store_f32<V>(p.ds0 + static_cast<int64_t>(s) * p.W + c0, cc);
          }
        }
      };
      if (tile.any) rows_out(Yes{}); else rows_out(No{});
    }
    fetch(sm.tile[slot2], buf);   // the buffer has been read to the end
    tile = next;
    slot = slot1;
  }
  copy_wait<0>();
}

template <typename T>
__global__ void __launch_bounds__(256) rec_step_kernel(const T* __restrict__ x, const T* __restrict__ f,
                                                       T* __restrict__ out, float* __restrict__ state, int64_t n,
                                                       int tied) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const float xv = load_elem<T>(x, i);
    float2 a, keep;
    gates<T>(make_float2(load_elem<T>(f, i), 0.f), a, keep);
    const float h = fmaf(a.x, state[i], tied ? keep.x * xv : xv);
    state[i] = h;
    store_elem<T>(out, i, h);
  }
}

using ForwardB = Shape<uint16_t, FSV, FSC, FSR>;
using BackwardB = Shape<uint16_t, BSV, BSC, BSR>;
using VectorF = Shape<float, 4, 8, 4>;       // 128 rows x 32 channels
using ScalarB = Shape<uint16_t, 1, 32, 16>;  // 128 rows x 32 channels
using ScalarF = Shape<float, 1, 32, 16>;

bool vectors(int W, la_dtype dt) { return W % (dt == LA_BF16 ? 8 : 4) == 0; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

template <class K> cudaError_t launch_kernel(K kernel, unsigned grid, size_t smem, const RecArgs& p, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <class S> cudaError_t launch_forward(RecArgs p, cudaStream_t stream) {
  p.nblocks = (p.W + S::C - 1) / S::C;
  const int64_t tiles = static_cast<int64_t>(p.ntiles) * p.nblocks, most = FB * static_cast<int64_t>(sm_count());
  const unsigned grid = static_cast<unsigned>(tiles < most ? tiles : most);
  const size_t smem = sizeof(Smem<S, 2, 2>);
  return p.tied ? launch_kernel(rec_forward_kernel<S, true>, grid, smem, p, stream)
                : launch_kernel(rec_forward_kernel<S, false>, grid, smem, p, stream);
}
template <class S> cudaError_t launch_backward(RecArgs p, cudaStream_t stream) {
  p.nblocks = (p.W + S::C - 1) / S::C;
  const int64_t tiles = static_cast<int64_t>(p.ntiles) * p.nblocks, most = BB * static_cast<int64_t>(sm_count());
  const unsigned grid = static_cast<unsigned>(tiles < most ? tiles : most);
  const size_t smem = sizeof(SmemBack<S, 3, 2>);
  return p.tied ? launch_kernel(rec_backward_kernel<S, true>, grid, smem, p, stream)
                : launch_kernel(rec_backward_kernel<S, false>, grid, smem, p, stream);
}

// Workspace: [error record] [ticket] [tiles' (A, H)] [states after the tiles] (these three set for
// each walk) [a copy of the states that a call in place overwrites] [backward: checkpoints, for a
// call that was given none].
struct RecLayout {
  int ntiles;
  size_t ctl, agg, inc, copy, ck, total;
};
RecLayout rec_layout(int nseq, int64_t tokens, int W, la_dtype dt, bool backward) {
  RecLayout l{};
  const size_t cols = (static_cast<size_t>(W) + 63) / 64 * 64;   // whole tiles of 32 or 64 channels
  l.ntiles = static_cast<int>((tokens + kCkRows - 1) / kCkRows);
  const size_t cells = l.ntiles * cols;
  const bool chain = l.ntiles > 1;
  l.ctl = 256;
  l.agg = chain ? up256(sizeof(uint64_t) * cells) : 0;
  l.inc = chain ? up256(sizeof(unsigned int) * cells) : 0;
  l.copy = up256(sizeof(float) * static_cast<size_t>(nseq) * W);
  l.ck = backward ? up256(sizeof(float) * static_cast<size_t>((tokens + kCkRows - 1) / kCkRows) * W) : 0;
  l.total = sizeof(ErrRec) + l.ctl + l.agg + l.inc + l.copy + l.ck;
  return l;
}

// One walk over the tiles, forward or backward in time.
cudaError_t launch_rec(RecArgs p, const RecLayout& l, la_dtype dt, bool backward, void* workspace,
                       cudaStream_t stream) {
  char* base = static_cast<char*>(workspace) + sizeof(ErrRec);
  p.ntiles = l.ntiles;
  p.ticket = reinterpret_cast<unsigned int*>(base);
  p.agg = reinterpret_cast<uint64_t*>(base + l.ctl);
  p.inc = reinterpret_cast<unsigned int*>(base + l.ctl + l.agg);
  // Where the states are updated in place, a tile may write what another still reads: from a copy.
  const float*& from = backward ? p.ds1 : p.s0;
  const float* to = backward ? p.ds0 : p.s1;
  const size_t bytes = sizeof(float) * static_cast<size_t>(p.nseq) * p.W;
  const uintptr_t fi = reinterpret_cast<uintptr_t>(from), ti = reinterpret_cast<uintptr_t>(to);
  cudaError_t e = cudaSuccess;
  if (p.tokens == 0) {   // no rows: the states pass through
    if (!to || from == to) return e;
    float* dst = backward ? p.ds0 : p.s1;
    return from ? cudaMemcpyAsync(dst, from, bytes, cudaMemcpyDeviceToDevice, stream)
                : cudaMemsetAsync(dst, 0, bytes, stream);
  }
  if (from && to && fi < ti + bytes && ti < fi + bytes) {
    float* copy = reinterpret_cast<float*>(base + l.ctl + l.agg + l.inc);
    e = cudaMemcpyAsync(copy, from, bytes, cudaMemcpyDeviceToDevice, stream);
    from = copy;
  }
  if (e == cudaSuccess && l.ntiles > 1) e = cudaMemsetAsync(p.ticket, 0xFF, l.ctl + l.agg + l.inc, stream);
  if (e != cudaSuccess) return e;
  const bool vec = vectors(p.W, dt);
  if (backward)
    return dt == LA_BF16 ? (vec ? launch_backward<BackwardB>(p, stream) : launch_backward<ScalarB>(p, stream))
                         : (vec ? launch_backward<VectorF>(p, stream) : launch_backward<ScalarF>(p, stream));
  return dt == LA_BF16 ? (vec ? launch_forward<ForwardB>(p, stream) : launch_forward<ScalarB>(p, stream))
                       : (vec ? launch_forward<VectorF>(p, stream) : launch_forward<ScalarF>(p, stream));
}

la_status common_rec(RecArgs& p, la_dtype dt, la_input_mode mode, void* workspace, size_t ws_bytes, bool backward,
                     cudaStream_t stream) {
  if ((dt != LA_F32 && dt != LA_BF16) || (mode != LA_INPUT_PLAIN && mode != LA_INPUT_TIED)) return LA_ERR_INVALID_ARG;
  if (p.nseq < 1 || p.W < 1 || p.tokens < 0) return LA_ERR_INVALID_ARG;
  if (p.tokens > INT32_MAX) return LA_ERR_UNSUPPORTED;
  if (p.tokens > 0) {
    const void* in[3] = {p.x, p.f, p.dout};
    void* out[2] = {backward ? p.dx : p.out, p.df};
    const int nin = backward ? 3 : 2, nout = backward ? 2 : 1;
    for (int i = 0; i < nin; ++i)
      if (!in[i] || !aligned16(in[i])) return LA_ERR_INVALID_ARG;
    for (int o = 0; o < nout; ++o) {
      if (!out[o] || !aligned16(out[o])) return LA_ERR_INVALID_ARG;
      for (int i = 0; i < nin; ++i)
        if (out[o] == in[i]) return LA_ERR_INVALID_ARG;
    }
    if (backward && p.dx == p.df) return LA_ERR_INVALID_ARG;
  }
  for (const void* s : {static_cast<const void*>(p.s0), static_cast<const void*>(p.s1),
                        static_cast<const void*>(p.ds0), static_cast<const void*>(p.ds1),
                        static_cast<const void*>(p.ck)})
    if (s && !aligned16(s)) return LA_ERR_INVALID_ARG;
  const RecLayout l = rec_layout(p.nseq, p.tokens, p.W, dt, backward);
  if (!workspace || !aligned256(workspace) || ws_bytes < l.total) return LA_ERR_INVALID_ARG;
  // tickets count tiles of 32 channels and are drawn two ahead by every CTA
  if (static_cast<int64_t>(l.ntiles) * ((p.W + 31) / 32) > INT32_MAX - 65536) return LA_ERR_UNSUPPORTED;
  p.err = static_cast<ErrRec*>(workspace);
  p.tied = mode == LA_INPUT_TIED;
  cudaError_t e = cudaSuccess;
  if (backward && !p.ck) {   // the forward's walk without its output
    RecArgs r = p;
    r.s1 = nullptr;
    r.ck = p.ck = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.total - l.ck);
    e = launch_rec(r, l, dt, false, workspace, stream);
  }
  if (e == cudaSuccess) e = launch_rec(p, l, dt, backward, workspace, stream);
  if (e != cudaSuccess) return LA_ERR_CUDA;
  set_last_path(backward ? "recurrence-backward" : "recurrence");
  return LA_OK;
}

RecArgs forward_args(const void* x, const void* f, void* out, const float* state_in, float* state_out,
                     float* checkpoints) {
  RecArgs p{};
  p.x = x; p.f = f; p.out = out;
  p.s0 = state_in; p.s1 = state_out; p.ck = checkpoints;
  return p;
}
RecArgs backward_args(const void* x, const void* f, const void* dout, void* dx, void* df, const float* state_in,
                      const float* dstate_out, float* dstate_in, const float* checkpoints) {
  RecArgs p{};
  p.x = x; p.f = f; p.dout = dout; p.dx = dx; p.df = df;
  p.s0 = state_in; p.ds1 = dstate_out; p.ds0 = dstate_in; p.ck = const_cast<float*>(checkpoints);
  return p;
}

}  // namespace
}  // namespace la

extern "C" {

la_status lightning_attn_gated_recurrence(const void* x, const void* f, void* out, const float* state_in,
                                          float* state_out, float* checkpoints, int B, int T, int W, la_dtype dtype,
                                          la_input_mode input_mode, void* workspace, size_t workspace_bytes,
                                          la_stream_t stream) {
  if (B < 1 || T < 0) return LA_ERR_INVALID_ARG;
  la::RecArgs p = la::forward_args(x, f, out, state_in, state_out, checkpoints);
  p.nseq = B; p.T = T; p.W = W; p.tokens = static_cast<int64_t>(B) * T;
  return la::common_rec(p, dtype, input_mode, workspace, workspace_bytes, false,
                        reinterpret_cast<cudaStream_t>(stream));
}

la_status lightning_attn_gated_recurrence_varlen(const void* x, const void* f, void* out, const float* state_in,
                                                 float* state_out, float* checkpoints, const int* cu_seqlens,
                                                 int num_seqs, int total_tokens, int W, la_dtype dtype,
                                                 la_input_mode input_mode, void* workspace, size_t workspace_bytes,
                                                 la_stream_t stream) {
  if (!cu_seqlens || !la::aligned16(cu_seqlens)) return LA_ERR_INVALID_ARG;
  la::RecArgs p = la::forward_args(x, f, out, state_in, state_out, checkpoints);
  p.cu = cu_seqlens; p.nseq = num_seqs; p.W = W; p.tokens = total_tokens;
  return la::common_rec(p, dtype, input_mode, workspace, workspace_bytes, false,
                        reinterpret_cast<cudaStream_t>(stream));
}

la_status lightning_attn_gated_recurrence_backward(const void* x, const void* f, const void* dout, void* dx, void* df,
                                                   const float* state_in, const float* dstate_out, float* dstate_in,
                                                   const float* checkpoints, int B, int T, int W, la_dtype dtype,
                                                   la_input_mode input_mode, void* workspace, size_t workspace_bytes,
                                                   la_stream_t stream) {
  if (B < 1 || T < 0) return LA_ERR_INVALID_ARG;
  la::RecArgs p = la::backward_args(x, f, dout, dx, df, state_in, dstate_out, dstate_in, checkpoints);
  p.nseq = B; p.T = T; p.W = W; p.tokens = static_cast<int64_t>(B) * T;
  return la::common_rec(p, dtype, input_mode, workspace, workspace_bytes, true,
                        reinterpret_cast<cudaStream_t>(stream));
}

la_status lightning_attn_gated_recurrence_backward_varlen(const void* x, const void* f, const void* dout, void* dx,
                                                          void* df, const float* state_in, const float* dstate_out,
                                                          float* dstate_in, const float* checkpoints,
                                                          const int* cu_seqlens, int num_seqs, int total_tokens, int W,
                                                          la_dtype dtype, la_input_mode input_mode, void* workspace,
                                                          size_t workspace_bytes, la_stream_t stream) {
  if (!cu_seqlens || !la::aligned16(cu_seqlens)) return LA_ERR_INVALID_ARG;
  la::RecArgs p = la::backward_args(x, f, dout, dx, df, state_in, dstate_out, dstate_in, checkpoints);
  p.cu = cu_seqlens; p.nseq = num_seqs; p.W = W; p.tokens = total_tokens;
  return la::common_rec(p, dtype, input_mode, workspace, workspace_bytes, true,
                        reinterpret_cast<cudaStream_t>(stream));
}

la_status lightning_attn_gated_recurrence_step(const void* x, const void* f, void* out, float* state, int B, int W,
                                               la_dtype dtype, la_input_mode input_mode, la_stream_t stream) {
  if (B < 1 || W < 1 || (dtype != LA_F32 && dtype != LA_BF16) ||
      (input_mode != LA_INPUT_PLAIN && input_mode != LA_INPUT_TIED))
    return LA_ERR_INVALID_ARG;
  for (const void* t : {x, f, static_cast<const void*>(out), static_cast<const void*>(state)})
    if (!t || !la::aligned16(t)) return LA_ERR_INVALID_ARG;
  if (out == x || out == f) return LA_ERR_INVALID_ARG;
  const int64_t n = static_cast<int64_t>(B) * W;
  const int64_t blocks = (n + 255) / 256;
  const unsigned grid = static_cast<unsigned>(blocks < 65535 ? blocks : 65535);
  const int tied = input_mode == LA_INPUT_TIED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == LA_BF16)
    la::rec_step_kernel<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(x),
                                                        static_cast<const uint16_t*>(f),
                                                        static_cast<uint16_t*>(out), state, n, tied);
  else
    la::rec_step_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(x), static_cast<const float*>(f),
                                                     static_cast<float*>(out), state, n, tied);
  if (cudaGetLastError() != cudaSuccess) return LA_ERR_CUDA;
  la::set_last_path("recurrence-step");
  return LA_OK;
}

size_t lightning_attn_gated_recurrence_workspace_size(int num_seqs, int total_tokens, int W, la_dtype dtype,
                                                      int backward) {
  if (num_seqs < 1 || total_tokens < 0 || W < 1 || (dtype != LA_F32 && dtype != LA_BF16)) return 0;
  return la::rec_layout(num_seqs, total_tokens, W, dtype, backward != 0).total;
}

}  // extern "C"
