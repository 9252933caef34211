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
// one that runs has been started and never waits for a later one.  A warp looks back over the
// tiles before its own until it finds one whose state after the last row is known, and folds the
// (A, H) between from there, oldest first.  That fold does the same operations in the same
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

struct RecArgs {
  const void *x, *f, *dout;
  void *out, *dx, *df;
  const float *s0, *ds1;
  float *s1, *ds0, *ck;
  const int* cu;
  int nseq, T, W, tied;
  int64_t tokens;
  ErrRec* err;
  // Chain between the tiles (more than one in time): cleared for each call.
  int ntiles, nblocks;          // in time, across the channels
  unsigned int* ticket;         // [0]: next tile; [1]: a wait ran out, everybody gives up
  unsigned int* flags;          // [ntiles][nblocks * C / 32]
  float2* agg;                  // [ntiles][nblocks * C]: (A, H) of the tile
  float* inc;                   // [ntiles][nblocks * C]: state after the tile
};

// a = sigmoid(f) and 1 - a = sigmoid(-f), each without cancellation: with e = exp(-|f|) in
// [0, 1], the larger of the two is 1 / (1 + e) and the smaller e / (1 + e).
struct Gate {
  float a, keep;
};
__device__ __forceinline__ Gate gate_of(float f) {
  const float e = expf(-fabsf(f));
  const float big = 1.0f / (1.0f + e), small = e * big;
  return f >= 0.0f ? Gate{big, small} : Gate{small, big};
}

// V consecutive channels of one row, as loaded.
template <typename T, int V> struct Pack;
template <> struct Pack<uint16_t, 8> {
  uint4 r;
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
  __device__ __forceinline__ static Pack from(const float* o) {
    return Pack{make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                           pack_bf16x2(o[6], o[7]))};
  }
};
template <> struct Pack<float, 4> {
  float4 r;
  __device__ __forceinline__ float get(int i) const { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }
  __device__ __forceinline__ static Pack from(const float* o) { return Pack{make_float4(o[0], o[1], o[2], o[3])}; }
};
template <> struct Pack<uint16_t, 1> {
  uint16_t r;
  __device__ __forceinline__ float get(int) const { return bf16_bits_to_f32(r); }
  __device__ __forceinline__ static Pack from(const float* o) { return Pack{f32_to_bf16_bits(o[0])}; }
};
template <> struct Pack<float, 1> {
  float r;
  __device__ __forceinline__ float get(int) const { return r; }
  __device__ __forceinline__ static Pack from(const float* o) { return Pack{o[0]}; }
};
template <int V> __device__ __forceinline__ void load_f32(const float* p, float* o) {
  if constexpr (V == 1) {
    o[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 t = *reinterpret_cast<const float4*>(p + i);
      o[i] = t.x; o[i + 1] = t.y; o[i + 2] = t.z; o[i + 3] = t.w;
    }
  }
}
template <int V> __device__ __forceinline__ void store_f32(float* p, const float* o) {
  if constexpr (V == 1) {
    *p = o[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
  }
}

// CL threads side by side take V channels each; G = 256 / CL groups of them take R rows each.
template <typename T_, int V_, int CL_, int R_> struct Shape {
  using T = T_;
  static constexpr int V = V_, CL = CL_, R = R_;
  static constexpr int C = CL * V, G = kThreads / CL, L = G * R;
  static constexpr int NP = kThreads / C, GP = G / NP;   // the fold over groups: NP threads a channel
  static_assert(C % 32 == 0 && kThreads % C == 0 && G % NP == 0 && kCkRows % R == 0, "tile");
};

template <class S> struct Smem {
  float A[S::G][S::C], H[S::G][S::C];     // of each group; then H: the state entering it
  float pA[S::NP][S::C], pH[S::NP][S::C];
  float in[S::C];
  int start[S::L], end[S::L];             // sequence that starts (ends) at the row, or -1
  int reset[S::G], preset[S::NP];
  int ticket;
};

__device__ __forceinline__ unsigned int load_acquire(const unsigned int* p) {
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(unsigned int* p, unsigned int v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Rows of the packed batch that belong to a sequence: the first `limit` ones.
__device__ __forceinline__ int64_t row_limit(const RecArgs& p) {
  if (!p.cu) return p.tokens;
  const int64_t n = __ldg(p.cu + p.nseq);
  return n < 0 ? 0 : n < p.tokens ? n : p.tokens;
}

// Marks the rows of tile `j` where sequences start and end.  Ends with a barrier.
template <int L> __device__ __forceinline__ void mark_rows(const RecArgs& p, int64_t r0, int* start, int* end) {
  const int tid = threadIdx.x;
  if (!p.cu) {
    for (int i = tid; i < L; i += kThreads) {
      const int row = static_cast<int>(r0 + i);   // tokens <= INT32_MAX; rows behind them are marked in vain
      const int s = row / p.T, t = row - s * p.T;
      const bool in = r0 + i < p.tokens;
      start[i] = in && t == 0 ? s : -1;
      end[i] = in && t == p.T - 1 ? s : -1;
    }
    __syncthreads();
    return;
  }
  for (int i = tid; i < L; i += kThreads) start[i] = end[i] = -1;
  __syncthreads();
  int lo = 0, hi = p.nseq;   // first sequence whose rows end behind r0
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (__ldg(p.cu + m + 1) > r0) hi = m; else lo = m + 1;
  }
  for (int s = lo + tid; s < p.nseq; s += kThreads) {
    const int64_t a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1);
    if (a >= r0 + L) break;
    if (a < 0 || b <= a || b > p.tokens) continue;
    if (a >= r0) start[a - r0] = s;
    if (b - 1 >= r0 && b - 1 < r0 + L) end[b - 1 - r0] = s;
  }
  __syncthreads();
}

// Sequences without rows: their final state (gradient) is the initial (final) one.  Malformed
// offsets are reported.  The sequences are dealt out to the time tiles.
__device__ __forceinline__ void rowless_sequences(const RecArgs& p, int j, int c0, int cn, const float* from,
                                                  float* to) {
  if (!p.cu) return;
  for (int64_t s = static_cast<int64_t>(j) * kThreads + threadIdx.x; s < p.nseq;
       s += static_cast<int64_t>(p.ntiles) * kThreads) {
    const int a = __ldg(p.cu + s), b = __ldg(p.cu + s + 1);
    if (a < 0 || b < a || b > p.tokens || (s == 0 && a != 0)) {
      report(p.err, LA_ERR_DEVICE, SITE_VARLEN_CU, static_cast<unsigned>(s), 0);
    } else if (a == b && to) {
      for (int c = c0; c < c0 + cn && c < p.W; ++c) to[s * p.W + c] = from ? from[s * p.W + c] : 0.f;
    }
  }
}

// One warp, 32 channels: what enters tile `k` (k counts tiles in the order of the walk; tile
// -1 does not exist).  `sub`: the warp's column of flags; `c`: the lane's column of data.
__device__ __forceinline__ float look_back(const RecArgs& p, int k, int sub, int nsub, int64_t c, int64_t cols) {
  const int lane = threadIdx.x & 31;
  int base = k - 1, from = -1;
  const uint64_t t0 = globaltimer_ns(), limit = wait_limit_ns(p.err);
  for (unsigned int polls = 0;;) {
    const int i = base - lane;
    const unsigned int st = i >= 0 ? load_acquire(p.flags + static_cast<int64_t>(i) * nsub + sub) : 2u;
    const unsigned int known = __ballot_sync(0xffffffffu, st == 2u), open = __ballot_sync(0xffffffffu, st == 0u);
    const unsigned int near = known ? (known & (0u - known)) - 1u : 0xffffffffu;   // tiles nearer than a known one
    if ((open & near) == 0) {
      if (known) {
        from = base - (__ffs(known) - 1);
        break;
      }
      base -= 32;   // 32 tiles whose (A, H) is there: look further back
      continue;
    }
    if ((++polls & 63u) == 0) {
      if (load_acquire(p.ticket + 1)) break;
      if (globaltimer_ns() - t0 > limit) {
        if (lane == 0) {
          report(p.err, LA_ERR_TIMEOUT, SITE_RECURRENCE_CHAIN, static_cast<unsigned>(k), static_cast<unsigned>(sub));
          store_release(p.ticket + 1, 1u);
        }
        break;
      }
    }
  }
  __syncwarp();
  if (from < 0) return 0.f;
  float h = __ldcg(p.inc + from * cols + c);
  int i = from + 1;
  for (; i + 8 <= k; i += 8) {
    float2 t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) t[u] = __ldcg(p.agg + (i + u) * cols + c);
#pragma unroll
    for (int u = 0; u < 8; ++u) h = fmaf(t[u].x, h, t[u].y);
  }
  for (; i < k; ++i) {
    const float2 t = __ldcg(p.agg + i * cols + c);
    h = fmaf(t.x, h, t.y);
  }
  return h;
}

// The fold over the CTA's groups and, through the chain, over the tiles before it: on return
// sm.H[g] is what enters group g.  On entry sm.A, sm.H, sm.reset hold each group's (A, H) and
// whether a sequence starts in it, so that what enters it does not leave it (and is not
// multiplied: it may be infinite).  Nothing (0) enters the walk's first tile.
// BACK: groups and tiles are walked from the last to the first.
template <class S, bool BACK>
__device__ __forceinline__ void fold_groups(const RecArgs& p, Smem<S>& sm, int k, int cb) {
  constexpr int C = S::C, NP = S::NP, GP = S::GP, G = S::G;
  const int c = threadIdx.x % C, part = threadIdx.x / C;
  float A[GP], H[GP];
  float pa = 1.f, ph = 0.f;
  int pr = 0;
#pragma unroll
  for (int i = 0; i < GP; ++i) {
    const int g = BACK ? G - 1 - (part * GP + i) : part * GP + i;
    A[i] = sm.A[g][c];
    H[i] = sm.H[g][c];
    const int r = sm.reset[g];
    ph = r ? H[i] : fmaf(A[i], ph, H[i]);
    pa *= A[i];
    pr |= r;
  }
  sm.pA[part][c] = pa;
  sm.pH[part][c] = ph;
  if (c == 0) sm.preset[part] = pr;
  __syncthreads();
  if (part == 0) {   // whole warps: C is a multiple of 32
    const int64_t cols = static_cast<int64_t>(p.nblocks) * C, col = static_cast<int64_t>(cb) * C + c;
    const int nsub = static_cast<int>(cols / 32), sub = static_cast<int>(col / 32);
    const bool chain = p.ntiles > 1;
    float tA = 1.f, tH = 0.f;
    int tr = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      tH = sm.preset[i] ? sm.pH[i][c] : fmaf(sm.pA[i][c], tH, sm.pH[i][c]);
      tA *= sm.pA[i][c];
      tr |= sm.preset[i];
    }
    unsigned int* flag = p.flags + static_cast<int64_t>(k) * nsub + sub;
    const bool alone = tr || k == 0;   // what leaves the tile does not need the tiles before it
    float in = 0.f;
    if (chain) {
      if (alone) p.inc[k * cols + col] = tH;
      else p.agg[k * cols + col] = make_float2(tA, tH);
      __syncwarp();
      if ((c & 31) == 0) store_release(flag, alone ? 2u : 1u);
      if (k > 0) {
        in = look_back(p, k, sub, nsub, col, cols);
        if (!alone) {
          p.inc[k * cols + col] = fmaf(tA, in, tH);
          __syncwarp();
          if ((c & 31) == 0) store_release(flag, 2u);
        }
      }
    }
    sm.in[c] = in;
  }
  __syncthreads();
  float h = sm.in[c];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (i < part) h = sm.preset[i] ? sm.pH[i][c] : fmaf(sm.pA[i][c], h, sm.pH[i][c]);
#pragma unroll
  for (int i = 0; i < GP; ++i) {
    const int g = BACK ? G - 1 - (part * GP + i) : part * GP + i;
    sm.H[g][c] = h;
    h = sm.reset[g] ? H[i] : fmaf(A[i], h, H[i]);
  }
  __syncthreads();
}

template <class S, bool TIED> __global__ void __launch_bounds__(kThreads) rec_forward_kernel(RecArgs p) {
  using T = typename S::T;
  constexpr int V = S::V, R = S::R;
  __shared__ Smem<S> sm;
  const int tid = threadIdx.x, cl = tid % S::CL, g = tid / S::CL;
  if (tid == 0) sm.ticket = p.ntiles > 1 ? static_cast<int>(atomicAdd(p.ticket, 1u)) : static_cast<int>(blockIdx.x);
  __syncthreads();
  const int k = sm.ticket / p.nblocks, cb = sm.ticket % p.nblocks;
  const int64_t r0 = static_cast<int64_t>(k) * S::L, row0 = r0 + g * R;
  const int c0 = cb * S::C + cl * V;
  const bool in = c0 < p.W;
  const T* x = static_cast<const T*>(p.x) + row0 * p.W + c0;
  const T* f = static_cast<const T*>(p.f) + row0 * p.W + c0;
  Pack<T, V> xr[R], fr[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (in && row0 + i < p.tokens) {
      xr[i] = *reinterpret_cast<const Pack<T, V>*>(x + static_cast<int64_t>(i) * p.W);
      fr[i] = *reinterpret_cast<const Pack<T, V>*>(f + static_cast<int64_t>(i) * p.W);
    } else {
      xr[i] = fr[i] = Pack<T, V>{};
    }
  }
  const int64_t limit = row_limit(p);
  rowless_sequences(p, k, cb * S::C, S::C, p.s0, p.s1);
  if (r0 >= limit) return;   // no later tile has rows either
  mark_rows<S::L>(p, r0, sm.start, sm.end);

  float a[R][V], b[R][V], A[V], H[V];
  int reset = 0;
#pragma unroll
  for (int e = 0; e < V; ++e) { A[e] = 1.f; H[e] = 0.f; }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int s = sm.start[g * R + i];
    if (s >= 0) {
      reset = 1;
#pragma unroll
      for (int e = 0; e < V; ++e) H[e] = 0.f;
      if (p.s0 && in) load_f32<V>(p.s0 + static_cast<int64_t>(s) * p.W + c0, H);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const Gate q = gate_of(fr[i].get(e));
      const float xv = xr[i].get(e);
      a[i][e] = q.a;
      b[i][e] = TIED ? q.keep * xv : xv;
      H[e] = fmaf(a[i][e], H[e], b[i][e]);
      A[e] *= a[i][e];
    }
  }
  store_f32<V>(&sm.A[g][cl * V], A);
  store_f32<V>(&sm.H[g][cl * V], H);
  if (cl == 0) sm.reset[g] = reset;
  __syncthreads();
  fold_groups<S, false>(p, sm, k, cb);

  if (!in) return;
  float h[V];
  load_f32<V>(&sm.H[g][cl * V], h);
  T* out = p.out ? static_cast<T*>(p.out) + row0 * p.W + c0 : nullptr;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (row0 + i >= limit) break;
    const int s = sm.start[g * R + i], e1 = sm.end[g * R + i];
    if (s >= 0) {
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = 0.f;
      if (p.s0) load_f32<V>(p.s0 + static_cast<int64_t>(s) * p.W + c0, h);
    }
    if (p.ck && (row0 + i) % kCkRows == 0) store_f32<V>(p.ck + (row0 + i) / kCkRows * p.W + c0, h);
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = fmaf(a[i][e], h[e], b[i][e]);
    if (out) *reinterpret_cast<Pack<T, V>*>(out + static_cast<int64_t>(i) * p.W) = Pack<T, V>::from(h);
    if (e1 >= 0 && p.s1) store_f32<V>(p.s1 + static_cast<int64_t>(e1) * p.W + c0, h);
  }
}

template <class S, bool TIED> __global__ void __launch_bounds__(kThreads) rec_backward_kernel(RecArgs p) {
  using T = typename S::T;
  constexpr int V = S::V, R = S::R, G = S::G;
  static_assert(S::L == kCkRows, "a tile starts at a checkpoint");
  __shared__ Smem<S> sm;
  const int tid = threadIdx.x, cl = tid % S::CL, g = tid / S::CL;
  if (tid == 0) sm.ticket = p.ntiles > 1 ? static_cast<int>(atomicAdd(p.ticket, 1u)) : static_cast<int>(blockIdx.x);
  __syncthreads();
  const int k = sm.ticket / p.nblocks, cb = sm.ticket % p.nblocks;
  const int j = p.ntiles - 1 - k;   // the walk goes backwards in time
  const int64_t r0 = static_cast<int64_t>(j) * S::L, row0 = r0 + g * R;
  const int c0 = cb * S::C + cl * V;
  const bool in = c0 < p.W;
  const int64_t at = row0 * p.W + c0;
  Pack<T, V> xr[R], fr[R], dr[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t o = at + static_cast<int64_t>(i) * p.W;
    if (in && row0 + i < p.tokens) {
      xr[i] = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(p.x) + o);
      fr[i] = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(p.f) + o);
      dr[i] = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(p.dout) + o);
    } else {
      xr[i] = fr[i] = dr[i] = Pack<T, V>{};
    }
  }
  const int64_t limit = row_limit(p);
  rowless_sequences(p, j, cb * S::C, S::C, p.ds1, p.ds0);
  mark_rows<S::L>(p, r0, sm.start, sm.end);

  // Forward in time inside the tile: the state entering each group.
  float a[R][V], A[V], H[V];
  int reset = 0;
#pragma unroll
  for (int e = 0; e < V; ++e) { A[e] = 1.f; H[e] = 0.f; }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int s = sm.start[g * R + i];
    if (s >= 0) {
      reset = 1;
#pragma unroll
      for (int e = 0; e < V; ++e) H[e] = 0.f;
      if (p.s0 && in) load_f32<V>(p.s0 + static_cast<int64_t>(s) * p.W + c0, H);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const Gate q = gate_of(fr[i].get(e));
      const float xv = xr[i].get(e);
      a[i][e] = q.a;
      H[e] = fmaf(q.a, H[e], TIED ? q.keep * xv : xv);
      A[e] *= q.a;
    }
  }
  store_f32<V>(&sm.A[g][cl * V], A);
  store_f32<V>(&sm.H[g][cl * V], H);
  if (cl == 0) sm.reset[g] = reset;
  __syncthreads();
  if (tid < S::C) {   // one thread a channel, group by group
    const int c = cb * S::C + tid;
    float h = r0 < limit && c < p.W ? p.ck[static_cast<int64_t>(j) * p.W + c] : 0.f;
#pragma unroll 4
    for (int i = 0; i < G; ++i) {
      const float hi = sm.H[i][tid];
      sm.H[i][tid] = h;
      h = sm.reset[i] ? hi : fmaf(sm.A[i][tid], h, hi);
    }
  }
  __syncthreads();
  float prev[R][V], h[V];
  load_f32<V>(&sm.H[g][cl * V], h);
  // Backward in time: what each group adds to the flow into the state before it.
  float cc[V];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int s = sm.start[g * R + i];
    if (s >= 0) {
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = 0.f;
      if (p.s0 && in) load_f32<V>(p.s0 + static_cast<int64_t>(s) * p.W + c0, h);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      prev[i][e] = h[e];
      const float xv = xr[i].get(e);
      h[e] = fmaf(a[i][e], h[e], TIED ? gate_of(fr[i].get(e)).keep * xv : xv);
    }
  }
  reset = 0;
#pragma unroll
  for (int e = 0; e < V; ++e) cc[e] = 0.f;
#pragma unroll
  for (int i = R - 1; i >= 0; --i) {
    const int s = sm.end[g * R + i];
    if (s >= 0) {
      reset = 1;
#pragma unroll
      for (int e = 0; e < V; ++e) cc[e] = 0.f;
      if (p.ds1 && in) load_f32<V>(p.ds1 + static_cast<int64_t>(s) * p.W + c0, cc);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) cc[e] = a[i][e] * (dr[i].get(e) + cc[e]);
  }
  __syncthreads();
  store_f32<V>(&sm.H[g][cl * V], cc);
  if (cl == 0) sm.reset[g] = reset;
  __syncthreads();
  fold_groups<S, true>(p, sm, k, cb);

  if (!in) return;
  load_f32<V>(&sm.H[g][cl * V], cc);
#pragma unroll
  for (int i = R - 1; i >= 0; --i) {
    if (row0 + i >= limit) continue;
    const int s = sm.start[g * R + i], e1 = sm.end[g * R + i];
    if (e1 >= 0) {
#pragma unroll
      for (int e = 0; e < V; ++e) cc[e] = 0.f;
      if (p.ds1) load_f32<V>(p.ds1 + static_cast<int64_t>(e1) * p.W + c0, cc);
    }
    float dx[V], df[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float keep = gate_of(fr[i].get(e)).keep;
      const float G1 = dr[i].get(e) + cc[e];
      const float kg = keep * G1;
      dx[e] = TIED ? kg : G1;
      df[e] = kg * a[i][e] * (TIED ? prev[i][e] - xr[i].get(e) : prev[i][e]);
      cc[e] = a[i][e] * G1;
    }
    const int64_t o = at + static_cast<int64_t>(i) * p.W;
    *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(p.dx) + o) = Pack<T, V>::from(dx);
    *reinterpret_cast<Pack<T, V>*>(static_cast<T*>(p.df) + o) = Pack<T, V>::from(df);
    if (s >= 0 && p.ds0) store_f32<V>(p.ds0 + static_cast<int64_t>(s) * p.W + c0, cc);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) rec_step_kernel(const T* __restrict__ x, const T* __restrict__ f,
                                                       T* __restrict__ out, float* __restrict__ state, int64_t n,
                                                       int tied) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const float xv = load_elem<T>(x, i);
    const Gate g = gate_of(load_elem<T>(f, i));
    const float h = fmaf(g.a, state[i], tied ? g.keep * xv : xv);
    state[i] = h;
    store_elem<T>(out, i, h);
  }
}

using ShapeB8 = Shape<uint16_t, 8, 8, 4>;    // 128 rows x 64 channels
using ShapeF4 = Shape<float, 4, 16, 8>;      // 128 rows x 64 channels
using ShapeB1 = Shape<uint16_t, 1, 32, 16>;  // 128 rows x 32 channels
using ShapeF1 = Shape<float, 1, 32, 16>;

bool vectors(int W, la_dtype dt) { return W % (dt == LA_BF16 ? 8 : 4) == 0; }
int tile_channels(int W, la_dtype dt) { return vectors(W, dt) ? 64 : 32; }
constexpr int kTileRows = 128;

template <class S> cudaError_t launch_shape(const RecArgs& p, bool backward, cudaStream_t stream) {
  static_assert(S::L == kTileRows, "workspace layout");
  const unsigned grid = static_cast<unsigned>(p.ntiles) * static_cast<unsigned>(p.nblocks);
  if (!backward) {
    if (p.tied) rec_forward_kernel<S, true><<<grid, kThreads, 0, stream>>>(p);
    else rec_forward_kernel<S, false><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (p.tied) rec_backward_kernel<S, true><<<grid, kThreads, 0, stream>>>(p);
    else rec_backward_kernel<S, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace: [error record] [ticket, flags (cleared for each call)] [tiles' (A, H)] [states after
// the tiles] [a copy of the states that a call in place overwrites] [backward: checkpoints, for a
// call that was given none].
struct RecLayout {
  int ntiles, nblocks;
  size_t ctl, agg, inc, copy, ck, total;
};
RecLayout rec_layout(int nseq, int64_t tokens, int W, la_dtype dt, bool backward) {
  RecLayout l{};
  const int C = tile_channels(W, dt);
  l.ntiles = static_cast<int>((tokens + kTileRows - 1) / kTileRows);
  l.nblocks = (W + C - 1) / C;
  const size_t cells = static_cast<size_t>(l.ntiles) * l.nblocks * C;
  l.ctl = up256(256 + sizeof(unsigned int) * (cells / 32));
  l.agg = up256(sizeof(float2) * cells);
  l.inc = up256(sizeof(float) * cells);
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
  p.nblocks = l.nblocks;
  p.ticket = reinterpret_cast<unsigned int*>(base);
  p.flags = reinterpret_cast<unsigned int*>(base + 256);
  p.agg = reinterpret_cast<float2*>(base + l.ctl);
  p.inc = reinterpret_cast<float*>(base + l.ctl + l.agg);
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
  if (e == cudaSuccess && l.ntiles > 1) e = cudaMemsetAsync(p.ticket, 0, l.ctl, stream);
  if (e != cudaSuccess) return e;
  if (dt == LA_BF16)
    return vectors(p.W, dt) ? launch_shape<ShapeB8>(p, backward, stream) : launch_shape<ShapeB1>(p, backward, stream);
  return vectors(p.W, dt) ? launch_shape<ShapeF4>(p, backward, stream) : launch_shape<ShapeF1>(p, backward, stream);
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
  if (static_cast<int64_t>(l.ntiles) * l.nblocks > INT32_MAX) return LA_ERR_UNSUPPORTED;
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
