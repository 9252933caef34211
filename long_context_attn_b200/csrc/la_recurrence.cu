// Gated linear recurrence h_t = a_t h_{t-1} + b_t, a = sigmoid(f), b = x or (1 - a) x, channel
// by channel: forward, one-token step and backward (sm_100a).
//
// Rows t .. u of a channel act on the state that enters them as h -> A h + H, A the product of
// their gates; two neighbours compose to (A2 A1, A2 H1 + H2).  A CTA walks C channels of the
// packed rows in tiles of L rows, reading each once.  In a tile a thread takes R rows of two
// channels and folds them to (A, H), keeping their a and b in registers; the groups of a warp
// compose with shuffles, the warps through shared memory, and every thread folds all warps
// from the state that entered the tile, so that it has both the state entering its own rows and the
// one entering the next tile: one barrier a tile.  Then it walks its rows again and writes them.  A row
// that starts a sequence takes its state from state_in instead, so packed sequences need no CTAs of
// their own.
//
// Where the channels are too few to fill the GPU, a cluster of up to 16 CTAs walks them together,
// each CTA a tile of the round's.  The CTAs send the (A, H) of their tiles into one another's shared
// memory, where an mbarrier counts them; then every thread folds the round's tiles as it folds the
// warps.  A cluster's CTAs run at the same time, so every round arrives (the wait is bounded all the
// same), and the result is the same in every run.
//
// What bounds it: latency, with few warps to hide it.  The rows that a thread keeps take 128 registers, so an SM
// has 16 warps; 8192 x 8192 in bf16 is 24.4 instructions an element (the backward 40.8), which fill 57 % of the issue
// slots, with DRAM at 49 %: of 3.2 warps on a scheduler 1.07 are ready, the others wait for a fixed latency, the shared-memory
// and special-function queues, or the barrier.  131072 x 8192 bf16 takes 1.44 ms, 4.5 TB/s of 6.56; backward of 8192 x 8192 145 us,
// 4.6 TB/s; 8192 x 8192 in fp32, half the elements a byte, 146 us, 5.5 TB/s.  Pairs of channels share an
// instruction where the hardware has one; tiles in which a sequence starts or ends, which are few, run code of
// their own, so that the others' has no tests (231 us with them at 16384 x 8192, 166 without).  In clusters a sixth of
// the warps' time goes to waiting for a round's sums.
// The time follows the fullest SM: 2^27 bf16 values take 277 us at 5120 channels (160 CTAs on 148 SMs), 173 at 8192, 152 at
// 9472 (296 CTAs, two an SM), and 236 at 9504, where the 297th CTA starts when the others end.
//
// The backward walks time in reverse: with c_t = a_t (dout_t + c_{t+1}) what flows into the
// state before row t, rows act on the c that enters them from behind as c -> A c + C with the same
// A.  h is recomputed from the checkpoint that the tile's first row starts from.
#include "la_common.cuh"
#include "la_f32x2.cuh"

namespace la {

void set_last_path(const char* path);

namespace {

constexpr int kCkRows = LA_RECURRENCE_CHECKPOINT_ROWS;
constexpr int kMaxCluster = 16, kMaxBackCluster = 8;   // the backward's fill the shared memory of two CTAs an SM
// The error record's site of a round that did not arrive (the tensor-core kernels' are 1 to 8), and the
// fault that makes the first CTA of a walk in clusters send nothing, so that its cluster's waits must run
// out (theirs is 1).
constexpr unsigned int kSiteRound = 9, kInjectSilent = 2;
constexpr int kThreads = 256, kWarps = kThreads / 32;

struct RecArgs {
  const void *x, *f, *dout;
  void *out, *dx, *df;
  const float *s0, *ds1;
  float *s1, *ds0, *ck;
  const int* cu;
  int nseq, T, W, tied;
  int64_t tokens;
  ErrRec* err;
  int nblocks;   // across the channels
};

// a = sigmoid(f) = 1 / (1 + t) and keep = 1 - a = t / (1 + t) with t = exp(-f), neither by
// cancellation.  Two special-function operations an element, exp2 and the reciprocal, which the
// memory rate leaves room for.  bf16 gates take exp2 of the rounded product -f log2(e): t is
// then off by at most (4 + |f|) 2^-24, against the 2^-9 the gate itself is rounded to (with expf
// and an IEEE division the first tiled kernel spent 47 instructions an element and ran at 0.30
// of the HBM rate, instruction-bound); fp32 gates call expf.  A Newton-Raphson step
// brings the approximate reciprocal to a correctly rounded one in nearly all cases: with the approximate
// one alone, states that remember 1000 tokens were 3 times as far off as with an IEEE division.  t is
// held to 2^126 (f < -87.3), so that 1 / (1 + t) stays a normal number and keep = 1 there; taking
// 2^-126 away from it makes a 0 there and changes no a above 2^-101.  A NaN passes.
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
__device__ __forceinline__ float min_nan(float x, float most) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(most));
  return y;
}
template <typename T> __device__ __forceinline__ void gates(F2 f, F2& a, F2& keep) {
  F2 t;
  if constexpr (sizeof(T) == 2) {
    const float2 y = split(mul2(f, splat(-1.4426950408889634f)));
    t = make_f2(exp2_approx(min_nan(y.x, 126.0f)), exp2_approx(min_nan(y.y, 126.0f)));
  } else {
    const float2 w = split(f);
    t = make_f2(min_nan(expf(-w.x), 0x1p126f), min_nan(expf(-w.y), 0x1p126f));
  }
  const F2 d = fma2(t, splat(-1.0f), splat(-1.0f));   // -(1 + t)
  const float2 v = split(d);
  F2 r = make_f2(rcp_approx(-v.x), rcp_approx(-v.y));
  r = fma2(r, fma2(d, r, splat(1.0f)), r);
  keep = mul2(t, r);
  a = add2(r, splat(-0x1p-126f));
}

// A thread's two channels of one row in shared memory.
__device__ __forceinline__ F2 load_pair(const uint16_t* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return make_f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ F2 load_pair(const float* p) { return *reinterpret_cast<const F2*>(p); }

// Two channels in global memory, the first at c; VEC: rows are aligned to pairs and whole pairs are
// inside (c < W).  Otherwise one by one, those that are.
template <bool VEC> __device__ __forceinline__ F2 load_state(const float* p, int c, int W) {
  if constexpr (VEC) return *reinterpret_cast<const F2*>(p);
  return make_f2(p[0], c + 1 < W ? p[1] : 0.f);
}
template <bool VEC> __device__ __forceinline__ void store_pair(float* p, F2 pair, int c, int W) {
  if constexpr (VEC) {
    *reinterpret_cast<F2*>(p) = pair;
  } else {
    const float2 v = split(pair);
    p[0] = v.x;
    if (c + 1 < W) p[1] = v.y;
  }
}
template <bool VEC> __device__ __forceinline__ void store_pair(uint16_t* p, F2 pair, int c, int W) {
  if constexpr (VEC) {
    const float2 v = split(pair);
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y);
  } else {
    const float2 v = split(pair);
    p[0] = f32_to_bf16_bits(v.x);
    if (c + 1 < W) p[1] = f32_to_bf16_bits(v.y);
  }
}

// CL threads side by side take two channels each; the G groups of a CTA, GW in a warp, take R rows each.
// VEC: rows are made of whole 16-byte vectors.
template <typename T_, int CL_, int R_, bool VEC_> struct Shape {
  using T = T_;
  static constexpr int CL = CL_, C = 2 * CL, GW = 32 / CL, G = kWarps * GW, R = R_, L = G * R;
  static constexpr bool VEC = VEC_;
  static_assert(L % kCkRows == 0 && kCkRows % R == 0, "a tile starts at a checkpoint, which a thread's first row may be");
};

// MOST: CTAs of a cluster, at most (1: without the arrays that only clusters need).
template <class S, int NT, int MOST> struct Smem {
  typename S::T raw[2][NT][S::L][S::C];   // of this tile and the next; each warp's rows are its own
  float A[2][kWarps][S::C], H[2][kWarps][S::C];
  int cut[2][kWarps];                     // whether a sequence starts in the warp's rows
  int mark[S::L];                         // see mark_rows(); each warp's rows are its own
  ulonglong2 round[2][MOST][S::CL];       // (A, H) of the round's tiles, each sent here by its CTA
  int round_cut[2][MOST];
  uint64_t arrived[2];                    // mbarriers: all of a round is here
};
// The backward's: the same for what flows back, beside the states forward in the tile.
template <class S, int MOST> struct SmemBack : Smem<S, 3, MOST> {
  float Cc[2][kWarps][S::C];
  int ccut[2][kWarps];
};

template <class S, bool CLUSTER> using ForwardSmem = Smem<S, 2, CLUSTER ? kMaxCluster : 1>;
template <class S, bool CLUSTER> using BackwardSmem = SmemBack<S, CLUSTER ? kMaxBackCluster : 1>;

// A warp's rows of a tile into shared memory, not waited for; zeros outside the rows and channels.
template <class S, int NT, int MOST>
__device__ __forceinline__ void fetch_rows(const RecArgs& p, Smem<S, NT, MOST>& sm, int buf, int64_t r0, int c0, int64_t limit) {
  using T = typename S::T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* src[3] = {static_cast<const T*>(p.x), static_cast<const T*>(p.f), static_cast<const T*>(p.dout)};
  constexpr int kWarpRows = S::L / kWarps;
  if constexpr (S::VEC) {
    constexpr int kVec = 16 / sizeof(T), kPer = S::C / kVec, kStep = 32 / kPer;   // lanes a row, rows at once
    const int r = warp * kWarpRows + lane / kPer, c = lane % kPer * kVec;
    const bool col = c0 + c < p.W, all = r0 + S::L <= limit;
    if (all && !col) return;   // zero since the beginning
    const int64_t step = static_cast<int64_t>(kStep) * p.W;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const T* at = src[q] + (r0 + r) * p.W + c0 + c;
      const unsigned int d = static_cast<unsigned int>(__cvta_generic_to_shared(&sm.raw[buf][q][r][c]));
#pragma unroll
      for (int i = 0; i < kWarpRows; i += kStep, at += step) {
        if (all) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + i * S::C * static_cast<int>(sizeof(T))), "l"(at)
                       : "memory");
        } else {
          const bool in = col && r0 + r + i < limit;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + i * S::C * static_cast<int>(sizeof(T))),
                       "l"(in ? at : src[q]), "r"(in ? 16 : 0) : "memory");
        }
      }
    }
  } else {   // element by element, waited for
#pragma unroll 1
    for (int q = 0; q < NT; ++q) {
#pragma unroll 1
      for (int i = 0; i < kWarpRows; ++i) {
        const int r = warp * kWarpRows + i;
        for (int c = lane; c < S::C; c += 32)
          sm.raw[buf][q][r][c] = c0 + c < p.W && r0 + r < limit ? src[q][(r0 + r) * p.W + c0 + c] : T(0);
      }
    }
  }
}
// Zeros the buffers' columns outside the channels, which fetch_rows() then leaves alone (the caller's
// barrier follows).
template <class S, int NT, int MOST> __device__ __forceinline__ void zero_columns(const RecArgs& p, Smem<S, NT, MOST>& sm, int c0) {
  if (!S::VEC || c0 + S::C <= p.W) return;
  using T = typename S::T;
  T* raw = &sm.raw[0][0][0][0];
  for (int i = threadIdx.x; i < 2 * NT * S::L * S::C; i += kThreads)
    if (c0 + i % S::C >= p.W) raw[i] = T(0);
}
__device__ __forceinline__ void commit_rows() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The warp's rows of the tile fetched before the last one are there.
__device__ __forceinline__ void rows_here() {
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  __syncwarp();
}

// Rows of the packed batch that belong to a sequence: the first `limit` ones.
__device__ __forceinline__ int64_t row_limit(const RecArgs& p) {
  if (!p.cu) return p.tokens;
  const int64_t n = __ldg(p.cu + p.nseq);
  return n < 0 ? 0 : n < p.tokens ? n : p.tokens;
}

// The sequence a row is in: the first that ends behind the row, from `from` to `to`.  A whole warp asks:
// it looks at 32 sequences at once, and by halves only where the row is far ahead.
struct Sequence {
  int s;
  int64_t lo, hi;
};
__device__ __forceinline__ Sequence sequence_of(const RecArgs& p, int64_t row, int from, int to) {
  Sequence q;
  if (!p.cu) {
    q.s = static_cast<int>(static_cast<unsigned int>(row) / static_cast<unsigned int>(p.T));   // row < tokens <= INT32_MAX
    q.lo = static_cast<int64_t>(q.s) * p.T;
    q.hi = q.lo + p.T;
    return q;
  }
  const int lane = threadIdx.x & 31;
  int a = from, b = to;
  while (b - a > 128) {
    const int mid = (a + b) >> 1, near = a + 64;
    if (__ldg(p.cu + near) > row) b = near;
    else if (__ldg(p.cu + mid + 1) > row) b = mid;
    else a = mid + 1;
  }
  for (;; a += 32) {   // ends: behind the last sequence everything is
    const unsigned int behind = __ballot_sync(0xffffffffu, a + lane >= p.nseq || __ldg(p.cu + a + lane + 1) > row);
    if (behind) {
      a += __ffs(behind) - 1;
      break;
    }
  }
  q.s = a;
  q.lo = a < p.nseq ? __ldg(p.cu + a) : p.tokens;
  q.hi = a < p.nseq ? __ldg(p.cu + a + 1) : p.tokens;
  return q;
}
// Whether the tile at r0 needs marks; without, every row of it is in one sequence, and none is that
// sequence's first or last.  `q`: the sequence of the row r0.
template <class S> __device__ __forceinline__ bool marked(const Sequence& q, int64_t r0, int64_t limit) {
  return q.lo >= r0 || q.hi <= r0 + S::L || r0 + S::L > limit;
}
// Marks the warp's rows of a tile: 4 s where sequence s starts or ends, with bit 0 set where it starts and
// bit 1 where it ends; -1 elsewhere.  `q`: the sequence of the tile's first row.
constexpr int kStart = 1, kEnd = 2;
template <class S>
__device__ __forceinline__ void mark_rows(const RecArgs& p, int64_t r0, int64_t limit, const Sequence& q, int* mark) {
  constexpr int kWarpRows = S::L / kWarps;
  const int lane = threadIdx.x & 31, at = (threadIdx.x >> 5) * kWarpRows;
  const int64_t first = r0 + at;
  int* own = mark + at;
  __syncwarp();   // the warp has done with the tile before
  if (!p.cu) {
    for (int i = lane; i < kWarpRows; i += 32) {
      const unsigned int T = p.T, row = static_cast<unsigned int>(first + i), s = row / T, in = row - s * T;
      const int m = (in == 0 ? kStart : 0) | (in == T - 1 ? kEnd : 0);
      own[i] = m && first + i < limit ? static_cast<int>(s) << 2 | m : -1;
    }
    __syncwarp();
    return;
  }
  for (int i = lane; i < kWarpRows; i += 32) own[i] = -1;
  __syncwarp();
  const int64_t end = first + kWarpRows < limit ? first + kWarpRows : limit;
  for (int s = q.s + lane;; s += 32) {   // a sequence a lane
    int64_t lo = p.tokens, hi = p.tokens;
    if (s < p.nseq) {
      lo = __ldg(p.cu + s);
      hi = __ldg(p.cu + s + 1);
    }
    if (s < p.nseq && lo >= 0 && hi > lo && hi <= p.tokens) {
      const bool starts = lo >= first && lo < end, ends = hi > first && hi <= end;
      if (starts) own[lo - first] = s << 2 | kStart | (hi == lo + 1 ? kEnd : 0);
      if (ends && !(starts && hi == lo + 1)) own[hi - 1 - first] = s << 2 | kEnd;
    }
    // until a lane is behind the warp's rows (a malformed order may end this early, or not before the last)
    if (__any_sync(0xffffffffu, s >= p.nseq || lo >= end)) break;
  }
  __syncwarp();
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

template <bool VEC> __device__ __forceinline__ F2 state_or_zero(const float* states, int s, int c0, int W) {
  return states ? load_state<VEC>(states + static_cast<int64_t>(s) * W + c0, c0, W) : splat(0.f);
}

// Acts on h as a run of rows with (A, H) does; `cut`: a sequence starts in the run, so what enters it
// does not leave it (and is not multiplied by 0: it may be infinite).
__device__ __forceinline__ F2 act(int cut, F2 A, F2 H, F2 h) { return cut ? H : fma2(A, h, H); }

__device__ __forceinline__ F2 shift(F2 pair, int d, bool up) {
  const float2 v = split(pair);
  return up ? make_f2(__shfl_up_sync(0xffffffffu, v.x, d), __shfl_up_sync(0xffffffffu, v.y, d))
            : make_f2(__shfl_down_sync(0xffffffffu, v.x, d), __shfl_down_sync(0xffffffffu, v.y, d));
}
// Composes the groups of a warp: (A, H, cut) of the lane's group becomes that of it and all groups
// before it (BACK: behind it), and (eA, eH, ecut) is that of those without it.
template <int CL, bool BACK>
__device__ __forceinline__ void compose_warp(F2& A, F2& H, int& cut, F2& eA, F2& eH, int& ecut) {
  const int gw = (threadIdx.x & 31) / CL, g = BACK ? 32 / CL - 1 - gw : gw;
#pragma unroll
  for (int d = 1; d < 32 / CL; d *= 2) {
    const F2 uA = shift(A, d * CL, !BACK), uH = shift(H, d * CL, !BACK);
    const int ucut = BACK ? __shfl_down_sync(0xffffffffu, cut, d * CL) : __shfl_up_sync(0xffffffffu, cut, d * CL);
    if (g >= d) {
      H = act(cut, A, H, uH);
      A = mul2(A, uA);
      cut |= ucut;
    }
  }
  eA = splat(1.f);
  eH = splat(0.f);
  ecut = 0;
  if constexpr (CL < 32) {
    const F2 uA = shift(A, CL, !BACK), uH = shift(H, CL, !BACK);
    const int ucut = BACK ? __shfl_down_sync(0xffffffffu, cut, CL) : __shfl_up_sync(0xffffffffu, cut, CL);
    if (g > 0) {
      eA = uA;
      eH = uH;
      ecut = ucut;
    }
  }
}

// The cluster's CTAs.
__device__ __forceinline__ unsigned int cluster_rank() {
  unsigned int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned int cluster_size() {
  unsigned int n;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
// Only at a kernel's begin and end: its release waits for the global stores on their way.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned int shared_address(const void* p) {
  return static_cast<unsigned int>(__cvta_generic_to_shared(p));
}
// The place in the shared memory of CTA `rank` that `p` is in this one's.
__device__ __forceinline__ unsigned int at_rank(const void* p, unsigned int rank) {
  unsigned int r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(shared_address(p)), "r"(rank));
  return r;
}
// Stores into another CTA's shared memory that its mbarrier counts when they are there.
__device__ __forceinline__ void send(unsigned int to, F2 a, F2 b, unsigned int mbar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(to), "l"(a.v),
               "l"(b.v), "r"(mbar) : "memory");
}
__device__ __forceinline__ void send(unsigned int to, int v, unsigned int mbar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to), "r"(v), "r"(mbar)
               : "memory");
}
__device__ __forceinline__ void mbar_init(uint64_t* m) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_address(m)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* m, unsigned int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_address(m)), "r"(bytes) : "memory");
}
// Waits until the phase of that parity is over; false where the time limit of every device-side wait ran
// out (reported; the caller waits no more).
__device__ __forceinline__ bool mbar_wait(uint64_t* m, unsigned int parity, ErrRec* err) {
  uint64_t t0 = 0;
  for (unsigned int polls = 1;; ++polls) {
    unsigned int done;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done) : "r"(shared_address(m)), "r"(parity) : "memory");
    if (done) return true;
    if ((polls & 63u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > wait_limit_ns(err)) {
        report(err, LA_ERR_TIMEOUT, kSiteRound, blockIdx.x, 0);
        return false;
      }
    }
  }
}
// What a CTA keeps of its cluster through the rounds.
struct Rounds {
  unsigned int rank, size, n = 0;   // n: rounds so far
  bool waiting = true;              // until a wait ran out
  bool silent = false;              // sends nothing: its wait ran out (or a failure test says so)
};
// The end of a cluster's walk: nobody leaves while others may still send into its shared memory.  Who had
// every round has had all that was sent to it.  Where a wait ran out, sends may be on their way that nothing
// counts any more; all of them were issued before the barrier, so the CTA stays for another millisecond, a
// thousand times what they take.
__device__ __forceinline__ void leave_cluster(const Rounds& rounds) {
  cluster_barrier();
  if (rounds.waiting) return;
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
}

// Once every warp's (A, H) is in shared memory (H and cut: of the walk's direction): what enters this
// warp's rows, from what enters the round's tiles, `state`, which becomes what leaves them.
template <class S, bool CLUSTER, bool BACK, bool MARKED, class M>
__device__ __forceinline__ F2 fold_warps(M& sm, int buf, const float (*H)[S::C], const int* cut, int cl, F2& state,
                                         Rounds& rounds, ErrRec* err) {
  const int warp = threadIdx.x >> 5;
  if constexpr (!CLUSTER) {
    F2 h = state;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int w = BACK ? kWarps - 1 - i : i;
      if (w == warp) h = state;
      state = act(MARKED ? cut[w] : 0, load_pair(&sm.A[buf][w][2 * cl]), load_pair(&H[w][2 * cl]), state);
    }
    return h;
  } else {
    // the tile's (A, H), and that of the warps before this one
    F2 tA = splat(1.f), tH = splat(0.f), bA = tA, bH = tH;
    int tcut = 0, bcut = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int w = BACK ? kWarps - 1 - i : i, r = MARKED ? cut[w] : 0;
      if (w == warp) { bA = tA; bH = tH; bcut = tcut; }
      const F2 wA = load_pair(&sm.A[buf][w][2 * cl]);
      tH = act(r, wA, load_pair(&H[w][2 * cl]), tH);
      tA = mul2(tA, wA);
      tcut |= r;
    }
    const unsigned int rank = rounds.rank, size = rounds.size;
    uint64_t* arrived = &sm.arrived[buf];
    if (threadIdx.x == 0 && rounds.waiting) mbar_expect(arrived, size * (S::CL * 16 + 4));   // once a phase
    for (unsigned int to = rounds.silent ? size : warp; to < size; to += kWarps) {   // a warp a CTA
      if ((threadIdx.x & 31) < S::CL) {
        const unsigned int mbar = at_rank(arrived, to);
        send(at_rank(&sm.round[buf][rank][cl], to), tA, tH, mbar);
        if (cl == 0) send(at_rank(&sm.round_cut[buf][rank], to), tcut, mbar);
      }
    }
    // The buffers take turns: a CTA sends into this one again only after it has had the next round from
    // everybody, who sent that after reading this one.
    if (rounds.waiting && !mbar_wait(arrived, rounds.n >> 1 & 1u, err)) {
      rounds.waiting = false;
      rounds.silent = true;
    }
    ++rounds.n;
    __syncwarp();
    F2 h = state;   // entering the tile
#pragma unroll 4
    for (unsigned int i = 0; i < size; ++i) {
      if (i == rank) h = state;
      const ulonglong2 t = sm.round[buf][i][cl];
      state = act(sm.round_cut[buf][i], F2{t.x}, F2{t.y}, state);
    }
    return act(bcut, bA, bH, h);
  }
}

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

template <class S, bool TIED, bool CLUSTER, int BLOCKS>
__global__ void __launch_bounds__(kThreads, BLOCKS) rec_forward_kernel(RecArgs p) {
  using T = typename S::T;
  constexpr int R = S::R, L = S::L;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<ForwardSmem<S, CLUSTER>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cl = tid % S::CL, g = tid / S::CL;
  Rounds rounds;
  rounds.rank = CLUSTER ? cluster_rank() : 0;
  rounds.size = CLUSTER ? cluster_size() : 1;
  const int stride = static_cast<int>(rounds.size);   // tiles a round
  const int cb = blockIdx.x / stride, c0 = cb * S::C + 2 * cl;
  const bool in = c0 < p.W;
  const int64_t limit = row_limit(p);
  const int filled = static_cast<int>((limit + L - 1) / L);   // tiles with rows
  rowless_sequences(p, p.s0, p.s1);
  zero_columns(p, sm, cb * S::C);
  __syncthreads();
  int t = static_cast<int>(rounds.rank);
  auto fetch = [&](int tile, int buf) {
    if (tile < filled) fetch_rows(p, sm, buf, static_cast<int64_t>(tile) * L, cb * S::C, limit);
    commit_rows();   // a group for every call, so that they can be counted
  };
  fetch(t, 0);
  fetch(t + stride, 1);
  if (CLUSTER) {   // everybody's mbarriers are there
    if (tid == 0) {
      mbar_init(&sm.arrived[0]);
      mbar_init(&sm.arrived[1]);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    rounds.silent = blockIdx.x == 0 && p.err->inject == kInjectSilent;
    cluster_barrier();
  }
  Sequence seq{0, 0, 0};   // of the tile's first row
  F2 state = splat(0.f);   // entering the round's first tile
  // every CTA of a cluster goes through every round, with a tile that has rows or without
  for (int buf = 0; t - t % stride < filled; t += stride, buf ^= 1) {
    const int64_t r0 = static_cast<int64_t>(t) * L, row0 = r0 + g * R;
    const int* mark = sm.mark + g * R;
    const bool rows = t < filled;   // a CTA without a tile in the last round takes part with an empty one
    if (rows && seq.hi <= r0) seq = sequence_of(p, r0, seq.s, p.nseq);
    const bool now = !rows || marked<S>(seq, r0, limit);
    if (now) mark_rows<S>(p, r0, limit, seq, sm.mark);
    auto tile = [&](auto with_marks) {   // the marks' tests are kept out of the common case
      constexpr bool kMarked = decltype(with_marks)::value;
      const T* x = &sm.raw[buf][0][g * R][2 * cl];
      const T* f = &sm.raw[buf][1][g * R][2 * cl];
      rows_here();

      F2 a[R], b[R], A = splat(1.f), H = splat(0.f);
      int cut = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if constexpr (kMarked) {
          const int m = mark[i];
          if (m >= 0 && (m & kStart)) {
            cut = 1;
            H = state_or_zero<S::VEC>(in ? p.s0 : nullptr, m >> 2, c0, p.W);
          }
        }
        F2 keep;
        gates<T>(load_pair(f + i * S::C), a[i], keep);
        b[i] = load_pair(x + i * S::C);
        if (TIED) b[i] = mul2(keep, b[i]);
        H = fma2(a[i], H, b[i]);
        A = mul2(A, a[i]);
      }
      __syncwarp();   // the warp's rows have been read
      fetch(t + 2 * stride, buf);
      F2 eA, eH;
      int ecut;
      compose_warp<S::CL, false>(A, H, cut, eA, eH, ecut);
      if (lane >= 32 - S::CL) {
        *reinterpret_cast<F2*>(&sm.A[buf][warp][2 * cl]) = A;
        *reinterpret_cast<F2*>(&sm.H[buf][warp][2 * cl]) = H;
        if (lane == 31) sm.cut[buf][warp] = cut;
      }
      __syncthreads();
      F2 h = fold_warps<S, CLUSTER, false, kMarked>(sm, buf, sm.H[buf], sm.cut[buf], cl, state, rounds, p.err);
      if (in && r0 < limit) {
        h = act(ecut, eA, eH, h);
        if (p.ck && row0 % kCkRows == 0 && row0 < limit) {
          const int m = kMarked ? mark[0] : -1;
          const bool first = m >= 0 && (m & kStart);
          store_pair<S::VEC>(p.ck + row0 / kCkRows * p.W + c0, first ? state_or_zero<S::VEC>(p.s0, m >> 2, c0, p.W) : h, c0, p.W);
        }
        if (p.out) {   // else the checkpoints are all that is wanted
          // a base the whole CTA shares and 32-bit offsets from it (L * W < 2^31)
          T* out = static_cast<T*>(p.out) + r0 * p.W + cb * S::C;
          unsigned int at = static_cast<unsigned int>(g * R) * static_cast<unsigned int>(p.W) + 2 * cl;
#pragma unroll
          for (int i = 0; i < R; ++i, at += p.W) {
            if constexpr (kMarked) {
              if (row0 + i >= limit) break;
              const int m = mark[i];
              if (m >= 0 && (m & kStart)) h = state_or_zero<S::VEC>(p.s0, m >> 2, c0, p.W);
            }
            h = fma2(a[i], h, b[i]);
            store_pair<S::VEC>(out + at, h, c0, p.W);
            if constexpr (kMarked) {
              const int m = mark[i];
              if (m >= 0 && (m & kEnd) && p.s1) store_pair<S::VEC>(p.s1 + static_cast<int64_t>(m >> 2) * p.W + c0, h, c0, p.W);
            }
          }
        }
      }
    };
    if (now) tile(Yes{}); else tile(No{});
  }
  if (CLUSTER) leave_cluster(rounds);
}

template <class S, bool TIED, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2) rec_backward_kernel(RecArgs p) {
  using T = typename S::T;
  constexpr int R = S::R, L = S::L, Q = R < 8 ? R : 8, NQ = R / Q;   // states are recomputed Q rows at a time
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sm = *reinterpret_cast<BackwardSmem<S, CLUSTER>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cl = tid % S::CL, g = tid / S::CL;
  Rounds rounds;
  rounds.rank = CLUSTER ? cluster_rank() : 0;
  rounds.size = CLUSTER ? cluster_size() : 1;
  const int stride = static_cast<int>(rounds.size);
  const int cb = blockIdx.x / stride, c0 = cb * S::C + 2 * cl;
  const bool in = c0 < p.W;
  const int64_t limit = row_limit(p);
  const int filled = static_cast<int>((limit + L - 1) / L);
  rowless_sequences(p, p.ds1, p.ds0);
  zero_columns(p, sm, cb * S::C);
  __syncthreads();
  int k = static_cast<int>(rounds.rank);   // tiles are counted from the last
  auto fetch = [&](int tile, int buf) {
    if (tile < filled) fetch_rows(p, sm, buf, static_cast<int64_t>(filled - 1 - tile) * L, cb * S::C, limit);
    commit_rows();
  };
  fetch(k, 0);
  fetch(k + stride, 1);
  if (CLUSTER) {
    if (tid == 0) {
      mbar_init(&sm.arrived[0]);
      mbar_init(&sm.arrived[1]);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    rounds.silent = blockIdx.x == 0 && p.err->inject == kInjectSilent;
    cluster_barrier();
  }
  Sequence seq{p.nseq, p.tokens, 0};   // of the tile's first row
  F2 flow = splat(0.f);   // entering the round's first tile from behind
  for (int buf = 0; k - k % stride < filled; k += stride, buf ^= 1) {
    const bool rows = k < filled;   // a CTA without a tile in the last round takes part with an empty one
    const int64_t r0 = rows ? static_cast<int64_t>(filled - 1 - k) * L : limit, row0 = r0 + g * R;
    const int* mark = sm.mark + g * R;
    if (rows && seq.lo > r0) {
      int from = 0, to = seq.s;
      if (p.cu) {   // near the one before, mostly
        const int near = to > 62 ? to - 62 : 0;
        if (__ldg(p.cu + near) <= r0) from = near; else to = near;
      }
      seq = sequence_of(p, r0, from, to);
    }
    const bool now = !rows || marked<S>(seq, r0, limit);
    if (now) mark_rows<S>(p, r0, limit, seq, sm.mark);
    auto tile = [&](auto with_marks) {
      constexpr bool kMarked = decltype(with_marks)::value;
      const T* x = &sm.raw[buf][0][g * R][2 * cl];
      const T* f = &sm.raw[buf][1][g * R][2 * cl];
      const T* d = &sm.raw[buf][2][g * R][2 * cl];
      F2 hin = splat(0.f);   // the state entering the tile
      if (in && rows) hin = load_state<S::VEC>(p.ck + r0 / kCkRows * p.W + c0, c0, p.W);
      rows_here();

      // What the group's rows do to the state, and to the flow into the state before them: C grows with
      // each row by the row's own part, carried over the rows before it (and the row) by A.  Every Q rows,
      // what the rows so far do to the state is kept.
      F2 a[R], keep[R], A = splat(1.f), H = splat(0.f), C = splat(0.f), qA[NQ], qH[NQ];
      int cut = 0, ccut = 0;
      unsigned int qcut = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (i % Q == 0) {
          qA[i / Q] = A;
          qH[i / Q] = H;
          qcut |= static_cast<unsigned int>(cut) << (i / Q);
        }
        gates<T>(load_pair(f + i * S::C), a[i], keep[i]);
        A = mul2(A, a[i]);
        F2 v = load_pair(d + i * S::C);
        if constexpr (kMarked) {
          const int m = mark[i];
          const bool starts = m >= 0 && (m & kStart), ends = m >= 0 && (m & kEnd);
          if (starts) {
            cut = 1;
            H = state_or_zero<S::VEC>(in ? p.s0 : nullptr, m >> 2, c0, p.W);
          }
          if (!ccut) {   // rows behind the end of a sequence flow to no row before it
            if (ends) v = add2(v, state_or_zero<S::VEC>(in ? p.ds1 : nullptr, m >> 2, c0, p.W));
            C = fma2(A, v, C);
          }
          ccut |= ends;
        } else {
          C = fma2(A, v, C);
        }
        const F2 xv = load_pair(x + i * S::C);
        H = fma2(a[i], H, TIED ? mul2(keep[i], xv) : xv);
      }
      const F2 gA = A;   // the group's own
      F2 eA = splat(1.f), eH = splat(0.f), bA, bC;
      int ecut = 0, bcut;
      F2 wA = gA;
      compose_warp<S::CL, false>(wA, H, cut, eA, eH, ecut);
      compose_warp<S::CL, true>(A, C, ccut, bA, bC, bcut);
      if (lane < S::CL) {   // all groups, from the last
        *reinterpret_cast<F2*>(&sm.A[buf][warp][2 * cl]) = A;
        *reinterpret_cast<F2*>(&sm.Cc[buf][warp][2 * cl]) = C;
        if (lane == 0) sm.ccut[buf][warp] = ccut;
      }
      if (lane >= 32 - S::CL) {
        *reinterpret_cast<F2*>(&sm.H[buf][warp][2 * cl]) = H;
        if (lane == 31) sm.cut[buf][warp] = cut;
      }
      __syncthreads();
      F2 c = fold_warps<S, CLUSTER, true, kMarked>(sm, buf, sm.Cc[buf], sm.ccut[buf], cl, flow, rounds, p.err);
      if (in && rows) {
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
          if (w < warp) hin = act(kMarked ? sm.cut[buf][w] : 0, load_pair(&sm.A[buf][w][2 * cl]), load_pair(&sm.H[buf][w][2 * cl]), hin);
        hin = act(ecut, eA, eH, hin);
        c = act(bcut, bA, bC, c);
        T* dx = static_cast<T*>(p.dx) + r0 * p.W + cb * S::C;
        T* df = static_cast<T*>(p.df) + r0 * p.W + cb * S::C;
        unsigned int at = static_cast<unsigned int>(g * R + R - 1) * static_cast<unsigned int>(p.W) + 2 * cl;
#pragma unroll
        for (int q = NQ - 1; q >= 0; --q) {
          F2 h = act(qcut >> q & 1u, qA[q], qH[q], hin), prev[Q];
#pragma unroll
          for (int j = 0; j < Q; ++j) {
            const int i = q * Q + j;
            if constexpr (kMarked) {
              const int m = mark[i];
              if (m >= 0 && (m & kStart)) h = state_or_zero<S::VEC>(p.s0, m >> 2, c0, p.W);
            }
            const F2 xv = load_pair(x + i * S::C);
            prev[j] = TIED ? fma2(xv, splat(-1.f), h) : h;   // what the gate weighs against the input
            h = fma2(a[i], h, TIED ? mul2(keep[i], xv) : xv);
          }
#pragma unroll
          for (int j = Q - 1; j >= 0; --j, at -= p.W) {
            const int i = q * Q + j;
            if constexpr (kMarked) {
              if (row0 + i >= limit) continue;
              const int m = mark[i];
              if (m >= 0 && (m & kEnd)) c = state_or_zero<S::VEC>(p.ds1, m >> 2, c0, p.W);
            }
            const F2 G1 = add2(load_pair(d + i * S::C), c);
            c = mul2(a[i], G1);
            store_pair<S::VEC>(dx + at, TIED ? mul2(keep[i], G1) : G1, c0, p.W);
            store_pair<S::VEC>(df + at, mul2(mul2(keep[i], c), prev[j]), c0, p.W);
            if constexpr (kMarked) {
              const int m = mark[i];
              if (m >= 0 && (m & kStart) && p.ds0) store_pair<S::VEC>(p.ds0 + static_cast<int64_t>(m >> 2) * p.W + c0, c, c0, p.W);
            }
          }
        }
      }
      __syncwarp();   // the warp's rows have been read to the end
      fetch(k + 2 * stride, buf);
    };
    if (now) tile(Yes{}); else tile(No{});
  }
  if (CLUSTER) leave_cluster(rounds);
}

// One token: 14 bytes an element in bf16 (x, f, out, and the fp32 state both ways), nothing else to wait
// for: V elements a thread, as many threads as that takes.
template <typename T, int V>
__global__ void __launch_bounds__(256) rec_step_kernel(const T* __restrict__ x, const T* __restrict__ f,
                                                       T* __restrict__ out, float* __restrict__ state, int64_t n,
                                                       int tied) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * V;
  if (i >= n) return;
  if constexpr (V == 1) {
    F2 a, keep;
    gates<T>(make_f2(load_elem<T>(f, i), 0.f), a, keep);
    const float xv = load_elem<T>(x, i);
    const float h = fmaf(split(a).x, state[i], tied ? split(keep).x * xv : xv);
    state[i] = h;
    store_elem<T>(out, i, h);
  } else {
    F2 h[V / 2], fv[V / 2], xv[V / 2];
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 t = *reinterpret_cast<const float4*>(state + i + e);
      h[e / 2] = make_f2(t.x, t.y);
      h[e / 2 + 1] = make_f2(t.z, t.w);
    }
    if constexpr (sizeof(T) == 2) {
      const uint4 fr = *reinterpret_cast<const uint4*>(f + i), xr = *reinterpret_cast<const uint4*>(x + i);
      const uint32_t fw[4] = {fr.x, fr.y, fr.z, fr.w}, xw[4] = {xr.x, xr.y, xr.z, xr.w};
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        fv[e] = make_f2(__uint_as_float(fw[e] << 16), __uint_as_float(fw[e] & 0xFFFF0000u));
        xv[e] = make_f2(__uint_as_float(xw[e] << 16), __uint_as_float(xw[e] & 0xFFFF0000u));
      }
    } else {
      const float4 fr = *reinterpret_cast<const float4*>(f + i), xr = *reinterpret_cast<const float4*>(x + i);
      fv[0] = make_f2(fr.x, fr.y);
      fv[1] = make_f2(fr.z, fr.w);
      xv[0] = make_f2(xr.x, xr.y);
      xv[1] = make_f2(xr.z, xr.w);
    }
    float2 o[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      F2 a, keep;
      gates<T>(fv[e], a, keep);
      o[e] = split(fma2(a, h[e], tied ? mul2(keep, xv[e]) : xv[e]));
    }
#pragma unroll
    for (int e = 0; e < V; e += 4)
      *reinterpret_cast<float4*>(state + i + e) = make_float4(o[e / 2].x, o[e / 2].y, o[e / 2 + 1].x, o[e / 2 + 1].y);
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint4*>(out + i) = make_uint4(pack_bf16x2(o[0].x, o[0].y), pack_bf16x2(o[1].x, o[1].y),
                                                      pack_bf16x2(o[2].x, o[2].y), pack_bf16x2(o[3].x, o[3].y));
    else
      *reinterpret_cast<float4*>(out + i) = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
  }
}
template <typename T, int V>
cudaError_t launch_step(const void* x, const void* f, void* out, float* state, int64_t n, int tied, cudaStream_t stream) {
  const int64_t blocks = (n / V + 255) / 256;   // V divides n
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  rec_step_kernel<T, V><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(static_cast<const T*>(x), static_cast<const T*>(f),
                                                                         static_cast<T*>(out), state, n, tied);
  return cudaGetLastError();
}

bool vectors(int W, la_dtype dt) { return W % (dt == LA_BF16 ? 8 : 4) == 0; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  return n;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

template <class K>
cudaError_t launch_kernel(K kernel, int nblocks, int cluster, size_t smem, const RecArgs& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess && cluster > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(nblocks) * static_cast<unsigned>(cluster));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  c.attrs = attr;
  c.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, p);
}
// CTAs that walk a block of channels together, `blocks` of them fitting an SM: as many as there is room for, from three up
// (bf16, 131072 x 1024: 834 us alone, 512, 349, 269, 240 in clusters of 2, 3, 4, 8; in pairs where two would fit,
// 32768 x 4096 takes 202 us, 215 alone).  9 to 15 left part of the GPU idle (131072 x 1024: 374 us with 9), so it is 8 or 16.
// Room for all CTAs is not room for all clusters, which lie in one group of SMs each: 14 of 16 CTAs run at once in bf16, and 15
// blocks wait for one another (65536 x 480: 102 us, 76 in clusters of 8; 16 to 18 blocks: 102 against 110); likewise 94 to 98 blocks in
// threes (32768 x 3008: 214 us, 213 alone).
int cluster_for(int nblocks, int64_t tiles, int blocks, int most) {
  int fit = blocks * sm_count() / nblocks;
  if (fit > most) fit = most;
  int n = fit >= 16 ? 16 : fit > 8 ? 8 : fit;
  if (n > tiles) n = static_cast<int>(tiles);
  if (n > 8 && n < 16) n = 8;
  return n < 3 ? 1 : n;
}
// CLUSTERS: where there are few channels; false for a shape that is only taken where there are many.
template <class S, bool TIED, int BLOCKS, bool CLUSTERS> cudaError_t launch_forward(RecArgs p, cudaStream_t stream) {
  p.nblocks = (p.W + S::C - 1) / S::C;
  if constexpr (CLUSTERS) {
    const int cluster = cluster_for(p.nblocks, (p.tokens + S::L - 1) / S::L, BLOCKS, kMaxCluster);
    if (cluster > 1)
      return launch_kernel(rec_forward_kernel<S, TIED, true, BLOCKS>, p.nblocks, cluster, sizeof(ForwardSmem<S, true>), p, stream);
  }
  return launch_kernel(rec_forward_kernel<S, TIED, false, BLOCKS>, p.nblocks, 1, sizeof(ForwardSmem<S, false>), p, stream);
}
template <class S, bool TIED> cudaError_t launch_backward(RecArgs p, cudaStream_t stream) {
  p.nblocks = (p.W + S::C - 1) / S::C;
  static_assert(sizeof(BackwardSmem<S, true>) <= 113 * 1024, "two CTAs an SM");
  const int cluster = cluster_for(p.nblocks, (p.tokens + S::L - 1) / S::L, 2, kMaxBackCluster);
  return cluster > 1 ? launch_kernel(rec_backward_kernel<S, TIED, true>, p.nblocks, cluster, sizeof(BackwardSmem<S, true>), p, stream)
                     : launch_kernel(rec_backward_kernel<S, TIED, false>, p.nblocks, 1, sizeof(BackwardSmem<S, false>), p, stream);
}
// bf16: tiles of 256 rows x 32 channels, 16 rows a thread; fp32, whose rows are twice the bytes: 128 x 32, 8
// rows a thread.  The fp32 forward takes 256 x 16 where blocks of 32 would be so few that three CTAs or more share one
// (up to 98 blocks on 148 SMs), whatever the length: three of its CTAs fit an SM and there are more blocks to share (65536 x 768:
// 140 us against 204; the backward, 319 against 262, does not), and 256 rows are one tile, not two (2048 channels: 200 rows 3.9 us
// against 5.8, 400 rows 6.1 against 6.8, 4000 rows 31 against 27).  Above 148 blocks of 16 it walks without clusters, where clusters of
// three with blocks of 32 would be faster from 4000 rows on (32768 x 2400: 284 us against 206).
template <typename T, bool VEC, bool TIED> cudaError_t launch_typed(const RecArgs& p, bool backward, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    using S = Shape<T, 16, 16, VEC>;
    return backward ? launch_backward<S, TIED>(p, stream) : launch_forward<S, TIED, 2, true>(p, stream);
  } else {
    using S = Shape<T, 16, 8, VEC>;
    if (backward) return launch_backward<S, TIED>(p, stream);
    if ((p.W + S::C - 1) / S::C * 3 <= 2 * sm_count()) return launch_forward<Shape<T, 8, 8, VEC>, TIED, 3, true>(p, stream);
    return launch_forward<S, TIED, 2, false>(p, stream);
  }
}
template <typename T> cudaError_t launch_walk(const RecArgs& p, bool vec, bool backward, cudaStream_t stream) {
  if (vec) return p.tied ? launch_typed<T, true, true>(p, backward, stream) : launch_typed<T, true, false>(p, backward, stream);
  return p.tied ? launch_typed<T, false, true>(p, backward, stream) : launch_typed<T, false, false>(p, backward, stream);
}

// Workspace: [error record] [a copy of the states that a call in place overwrites] [backward:
// checkpoints, for a call that was given none].
struct RecLayout {
  size_t copy, ck, total;
};
RecLayout rec_layout(int nseq, int64_t tokens, int W, bool backward) {
  RecLayout l{};
  l.copy = up256(sizeof(float) * static_cast<size_t>(nseq) * W);
  l.ck = backward ? up256(sizeof(float) * static_cast<size_t>((tokens + kCkRows - 1) / kCkRows) * W) : 0;
  l.total = sizeof(ErrRec) + l.copy + l.ck;
  return l;
}

// One walk over the rows, forward or backward in time.
cudaError_t launch_rec(RecArgs p, la_dtype dt, bool backward, void* workspace,
                       cudaStream_t stream) {
  char* base = static_cast<char*>(workspace) + sizeof(ErrRec);
  // Where the states are updated in place, a thread may write what another still reads: from a copy.
  const float*& from = backward ? p.ds1 : p.s0;
  float* to = backward ? p.ds0 : p.s1;
  const size_t bytes = sizeof(float) * static_cast<size_t>(p.nseq) * p.W;
  const bool pass = p.tokens == 0 && !p.cu;   // no rows: the states pass through (packed: in the kernel, which checks the offsets)
  if (pass && (!to || from == to)) return cudaSuccess;
  if (overlap(from, bytes, to, bytes)) {
    float* copy = reinterpret_cast<float*>(base);
    const cudaError_t e = cudaMemcpyAsync(copy, from, bytes, cudaMemcpyDeviceToDevice, stream);
    if (e != cudaSuccess) return e;
    from = copy;
  }
  if (pass)
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, stream) : cudaMemsetAsync(to, 0, bytes, stream);
  const bool vec = vectors(p.W, dt);
  return dt == LA_BF16 ? launch_walk<uint16_t>(p, vec, backward, stream) : launch_walk<float>(p, vec, backward, stream);
}

la_status common_rec(RecArgs& p, la_dtype dt, la_input_mode mode, void* workspace, size_t ws_bytes, bool backward,
                     cudaStream_t stream) {
  if ((dt != LA_F32 && dt != LA_BF16) || (mode != LA_INPUT_PLAIN && mode != LA_INPUT_TIED)) return LA_ERR_INVALID_ARG;
  if (p.nseq < 1 || p.W < 1 || p.tokens < 0) return LA_ERR_INVALID_ARG;
  // marks hold a sequence and two bits; offsets inside a tile are 32-bit
  if (p.tokens > INT32_MAX || p.nseq > (1 << 28) || p.W > (1 << 22)) return LA_ERR_UNSUPPORTED;
  if (p.tokens > 0) {
    for (const void* t : {p.x, p.f, static_cast<const void*>(backward ? p.dx : p.out)})
      if (!t || !aligned16(t)) return LA_ERR_INVALID_ARG;
    if (backward && (!p.dout || !aligned16(p.dout) || !p.df || !aligned16(p.df))) return LA_ERR_INVALID_ARG;
  }
  for (const void* s : {static_cast<const void*>(p.s0), static_cast<const void*>(p.s1),
                        static_cast<const void*>(p.ds0), static_cast<const void*>(p.ds1),
                        static_cast<const void*>(p.ck)})
    if (s && !aligned16(s)) return LA_ERR_INVALID_ARG;
  const RecLayout l = rec_layout(p.nseq, p.tokens, p.W, backward);
  if (!workspace || !aligned256(workspace) || ws_bytes < l.total) return LA_ERR_INVALID_ARG;
  // Rows and sequences are worked on in any order, so nothing that is written may meet anything else; but the
  // states the walk ends with may meet those it begins with, which are then read from a copy.
  const size_t rows = static_cast<size_t>(p.tokens) * p.W * (dt == LA_BF16 ? 2 : 4);
  const size_t states = sizeof(float) * static_cast<size_t>(p.nseq) * p.W;
  const size_t cks = sizeof(float) * static_cast<size_t>((p.tokens + kCkRows - 1) / kCkRows) * p.W;
  enum { kNever, kBegin, kEndOfWalk };
  const struct { const void* at; size_t bytes; bool written; int walk; } args[] = {
      {p.x, rows, false, kNever}, {p.f, rows, false, kNever}, {p.dout, rows, false, kNever},
      {p.cu, sizeof(int) * (static_cast<size_t>(p.nseq) + 1), false, kNever},
      {p.s0, states, false, backward ? kNever : kBegin}, {p.s1, states, true, kEndOfWalk},
      {p.ds1, states, false, kBegin}, {p.ds0, states, true, kEndOfWalk}, {p.ck, cks, !backward, kNever},
      {p.out, rows, true, kNever}, {p.dx, rows, true, kNever}, {p.df, rows, true, kNever},
      {workspace, l.total - (p.ck ? l.ck : 0), true, kNever}};   // room for checkpoints is not used where they are given
  for (const auto& w : args) {
    if (!w.written || !w.at) continue;
    for (const auto& t : args)
      if (t.at && &t != &w && !(w.walk == kEndOfWalk && t.walk == kBegin) && overlap(w.at, w.bytes, t.at, t.bytes))
        return LA_ERR_INVALID_ARG;
  }
  p.err = static_cast<ErrRec*>(workspace);
  p.tied = mode == LA_INPUT_TIED;
  cudaError_t e = cudaSuccess;
  if (backward && !p.ck) {   // the forward's walk without its output
    RecArgs r = p;
    r.s1 = nullptr;
    r.ck = p.ck = reinterpret_cast<float*>(static_cast<char*>(workspace) + l.total - l.ck);
    e = launch_rec(r, dt, false, workspace, stream);
  }
  if (e == cudaSuccess) e = launch_rec(p, dt, backward, workspace, stream);
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
  // the elements are independent: whole 16-byte vectors of the flat array where it is made of them
  const int64_t n = static_cast<int64_t>(B) * W;
  if (n > (int64_t(1) << 38)) return LA_ERR_UNSUPPORTED;
  const size_t row_bytes = static_cast<size_t>(n) * (dtype == LA_BF16 ? 2 : 4), state_bytes = static_cast<size_t>(n) * 4;
  for (const void* t : {x, f})
    if (la::overlap(out, row_bytes, t, row_bytes) || la::shifted(state, state_bytes, t, row_bytes)) return LA_ERR_INVALID_ARG;
  if (la::shifted(state, state_bytes, out, row_bytes)) return LA_ERR_INVALID_ARG;
  const int tied = input_mode == LA_INPUT_TIED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == LA_BF16 ? (n % 8 == 0 ? la::launch_step<uint16_t, 8>(x, f, out, state, n, tied, st)
                                     : la::launch_step<uint16_t, 1>(x, f, out, state, n, tied, st))
                       : (n % 4 == 0 ? la::launch_step<float, 4>(x, f, out, state, n, tied, st)
                                     : la::launch_step<float, 1>(x, f, out, state, n, tied, st));
  if (e != cudaSuccess) return LA_ERR_CUDA;
  la::set_last_path("recurrence-step");
  return LA_OK;
}

size_t lightning_attn_gated_recurrence_workspace_size(int num_seqs, int total_tokens, int W, la_dtype dtype,
                                                      int backward) {
  if (num_seqs < 1 || total_tokens < 0 || W < 1 || (dtype != LA_F32 && dtype != LA_BF16)) return 0;
  return la::rec_layout(num_seqs, total_tokens, W, backward != 0).total;
}

}  // extern "C"
