// Layer norm over rows of W values with the residual addition in front of it, forward and
// backward (sm_100a).
//
//   s = x + residual,  z = (s - mean) r,  r = 1 / sqrt(mean((s - mean)^2) + eps),  y = z w + b
//   g = dout w,  dx = r (g - mean(g) - z mean(g z)) + dsum,  dw = sum dout z,  db = sum dout
//
// A row stays in the registers of the G threads that share it (a warp, or a CTA) between its
// one read and its one write, so the deviations are squared after the mean is known and both
// passes touch memory once.  Memory is the forward's bound.  What keeps wide rows from it is the latency of a
// row's reductions with few rows on an SM, so CTAs stay and have the next rows on their way while
// they reduce one.  8192 x 8192 bf16 with the residual (537 MB): forward 121 us with a CTA a row, 104 with rows
// on their way and the weights read for each, 86 to 98 with the weights in registers (by the GPU; 82 at the copy rate).  The
// backward stays at those reductions' latency (one row on an SM at a time, DRAM at 59 %): 292, 148, 119 (two reductions a
// row instead of three, and the warps' sums added by shuffles), 113 (a warp's lanes divide the sums); its few parts
// of the sums take 11 us more to add, which is what few rows pay for (256 x 8192: 27 us, 3 at the copy rate).
#include "la_common.cuh"
#include "la_f32x2.cuh"

namespace la {
namespace {

// One thread's V consecutive values, as loaded (16 bytes, or one element), worked on in U pairs
// (V == 1: the second half of the pair is 0 and stays 0).
template <typename T, int V> struct Pack;
template <> struct Pack<uint16_t, 8> {
  uint4 r;
  __device__ __forceinline__ void unpack(F2* o) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = make_f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void pack(const F2* o) {
    const float2 a = split(o[0]), b = split(o[1]), c = split(o[2]), d = split(o[3]);
    r = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y), pack_bf16x2(d.x, d.y));
  }
};
template <> struct Pack<float, 4> {
  ulonglong2 r;
  __device__ __forceinline__ void unpack(F2* o) const { o[0].v = r.x; o[1].v = r.y; }
  __device__ __forceinline__ void pack(const F2* o) { r = make_ulonglong2(o[0].v, o[1].v); }
};
template <> struct Pack<uint16_t, 1> {
  uint16_t r;
  __device__ __forceinline__ void unpack(F2* o) const { o[0] = make_f2(bf16_bits_to_f32(r), 0.f); }
  __device__ __forceinline__ void pack(const F2* o) { r = f32_to_bf16_bits(split(o[0]).x); }
};
template <> struct Pack<float, 1> {
  float r;
  __device__ __forceinline__ void unpack(F2* o) const { o[0] = make_f2(r, 0.f); }
  __device__ __forceinline__ void pack(const F2* o) { r = split(o[0]).x; }
};
constexpr int pairs(int V) { return (V + 1) / 2; }

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V> __device__ __forceinline__ void store_pack(T* p, const F2* o) {
  Pack<T, V> k;
  k.pack(o);
  *reinterpret_cast<Pack<T, V>*>(p) = k;
}
// V fp32 values of the weight or bias (`fill` where there is none).
template <int V> __device__ __forceinline__ void load_w(const float* p, int c, float fill, F2* o) {
#pragma unroll
  for (int i = 0; i < pairs(V); ++i) o[i] = splat(fill);
  if (!p) return;
  if constexpr (V == 1) {
    o[0] = make_f2(__ldg(p + c), 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(p + c + i));
      o[i / 2] = make_f2(t.x, t.y);
      o[i / 2 + 1] = make_f2(t.z, t.w);
    }
  }
}

// N sums over the G threads of a row, in every one of them, in a fixed order.  A warp's lanes divide the sums among
// them, the half of a pair going on with one of it (6 shuffles for four sums, not 20), and so do the lanes that add the
// warps'.  `red` alternates between calls, so one barrier a call is enough.
using Sums = float[2][4][32];
__device__ __forceinline__ float divide_sums(float lower, float upper, int lanes) {
  const bool up = threadIdx.x & lanes;
  const float mine = up ? upper : lower, other = up ? lower : upper;
  return mine + __shfl_xor_sync(0xffffffffu, other, lanes);
}
template <int G, int N> __device__ __forceinline__ void row_sums(float (&v)[N], Sums& red, int& half) {
  static_assert(N == 1 || N == 2 || N == 4, "the lanes are divided by halves");
  constexpr int L = 32 / N;   // lanes a sum
  const int lane = threadIdx.x & 31;
  float a = v[0];
  if constexpr (N == 2) a = divide_sums(v[0], v[1], 16);
  if constexpr (N == 4) a = divide_sums(divide_sums(v[0], v[2], 16), divide_sums(v[1], v[3], 16), 8);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if constexpr (G > 32) {
    constexpr int NW = G / 32, S = NW < L ? NW : L;
    if (lane % L == 0) red[half][lane / L][threadIdx.x >> 5] = a;
    __syncthreads();
    a = red[half][lane / L][lane % S];
#pragma unroll
    for (int i = S; i < NW; i += S) a += red[half][lane / L][lane % S + i];
#pragma unroll
    for (int o = S / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    half ^= 1;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = N == 1 ? a : __shfl_sync(0xffffffffu, a, k * L);
}
__device__ __forceinline__ float both(F2 a) {
  const float2 v = split(a);
  return v.x + v.y;
}

// How a row lies in its G threads: NV vectors of V values each; FULL: exactly, so that no column is asked whether it is
// inside. It costs a second kernel of each vector form and gains on the widths that models mostly have
// (bf16, residual, forward and backward: 65536 x 1024 93 and 107 us against 121 and 120, 16384 x 4096 100 and 105 against 101 and
// 113, 8192 x 8192 99 and 112 against 97 and 125).
template <typename T_, int V_, int NV_, int G_, bool FULL_> struct Row {
  using T = T_;
  static constexpr int V = V_, NV = NV_, G = G_, U = pairs(V_);
  static constexpr bool FULL = FULL_;
  __device__ __forceinline__ static int column(int lane, int i) { return (lane + i * G) * V; }
  __device__ __forceinline__ static bool in(int lane, int i, int W) { return FULL || column(lane, i) < W; }
};

// A row held in registers becomes its deviations from a first mean, which is rounded: a sum of W values is off by
// up to 42 roundings of their size (32 of a thread's, 5 of a warp's, 5 of the warps').  8192 values of 1745.394 come out a
// last place beside their mean, and over sqrt(eps) = 0.0032 that is 0.077 in z, which should be 0.  So the
// mean of the deviations, `shift`, is taken off as well: their sum travels with that of their squares, and the variance is
// the squares' mean less shift^2.  What is left are 42 roundings of the deviations' size.
template <class R>
__device__ __forceinline__ void center(F2 (*v)[R::U], int W, int lane, Sums& red, int& half, float& sum, float& squares) {
  F2 a = splat(0.f);
#pragma unroll
  for (int i = 0; i < R::NV; ++i)
#pragma unroll
    for (int e = 0; e < R::U; ++e) a = add2(a, v[i][e]);
  float total[1] = {both(a)};
  row_sums<R::G>(total, red, half);
  const float mean = total[0] / static_cast<float>(W);
  const F2 minus = R::V == 1 ? make_f2(-mean, 0.f) : splat(-mean);
  F2 q = splat(0.f), d = splat(0.f);
#pragma unroll
  for (int i = 0; i < R::NV; ++i) {
    const bool in = R::in(lane, i, W);
#pragma unroll
    for (int e = 0; e < R::U; ++e) {
      v[i][e] = add2(v[i][e], minus);
      if (!in) v[i][e] = splat(0.f);
      d = add2(d, v[i][e]);
      q = fma2(v[i][e], v[i][e], q);
    }
  }
  sum = both(d);
  squares = both(q);
}
// 1 / sqrt(var + eps) of deviations with that mean (shift) and sum of squares. The difference of two close
// numbers may round below 0; squares beyond the range stay infinite (and a NaN a NaN).
__device__ __forceinline__ float inverse_std(float squares, float shift, float inv_w, float eps) {
  float var = squares * inv_w;
  if (var < INFINITY) var = fmaxf(fmaf(-shift, shift, var), 0.0f);
  return 1.0f / sqrtf(var + eps);
}

// Rows on their way into shared memory: SLOTS of them, NT tensors a row, in slots that only the
// thread that will use them touches (no barriers).  SLOTS == 0: a row is read when it is used.
template <class R, int TPB, int NT, int SLOTS> struct Ring {
  using T = typename R::T;
  using P = Pack<T, R::V>;
  static constexpr size_t kBytes = sizeof(P) * SLOTS * NT * R::NV * TPB;
  P* base;
  const T* src[NT];
  int W, lane;
  __device__ __forceinline__ P* slot(int n, int q, int i) const { return base + ((n * NT + q) * R::NV + i) * TPB + threadIdx.x; }
  __device__ __forceinline__ void fetch(int n, int64_t row, int64_t rows) const {
    if constexpr (SLOTS > 0) {
      if (row < rows) {
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const T* at = src[q] + row * W;
#pragma unroll
          for (int i = 0; i < R::NV; ++i) {
            if (R::in(lane, i, W)) {
              const unsigned int d = static_cast<unsigned int>(__cvta_generic_to_shared(slot(n, q, i)));
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(at + R::column(lane, i)) : "memory");
            }
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  // The row fetched SLOTS calls of fetch() ago is here.
  __device__ __forceinline__ void wait() const {
    if constexpr (SLOTS > 0) asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS > 0 ? SLOTS - 1 : 0) : "memory");
  }
  __device__ __forceinline__ P get(int n, int q, int i, int64_t row) const {
    if constexpr (SLOTS > 0) return *slot(n, q, i);
    return load_pack<T, R::V>(src[q] + row * W + R::column(lane, i));
  }
};

// A row in TPB / G groups of threads at a time; with SLOTS, by CTAs that stay, the next rows on their way.
// The weights and biases of wide rows are held, not read again: they are fp32, 64 KB a row of 8192, twice
// what the row itself is in bf16 (8192 x 8192 without residual: 88 us against 61).
template <class R, int TPB, bool RES, int SLOTS, int BLOCKS>
__global__ void __launch_bounds__(TPB, BLOCKS)
layer_norm_kernel(const typename R::T* x, const typename R::T* residual, const float* __restrict__ w,
                  const float* __restrict__ b, typename R::T* out, typename R::T* sum_out, int rows, int W, float eps) {
  using T = typename R::T;
  constexpr int V = R::V, NV = R::NV, U = R::U;
  constexpr bool kHold = SLOTS > 0 && NV * V <= 16;   // the thread's weights and biases stay in registers
  __shared__ Sums red;
  extern __shared__ __align__(16) unsigned char ring_smem[];
  const int lane = threadIdx.x % R::G;
  const float inv_w = 1.0f / static_cast<float>(W);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (TPB / R::G);
  int64_t row = static_cast<int64_t>(blockIdx.x) * (TPB / R::G) + threadIdx.x / R::G;
  Ring<R, TPB, RES ? 2 : 1, SLOTS> ring;
  ring.base = reinterpret_cast<Pack<T, V>*>(ring_smem);
  ring.src[0] = x;
  if (RES) ring.src[RES ? 1 : 0] = residual;
  ring.W = W;
  ring.lane = lane;
#pragma unroll
  for (int n = 0; n < SLOTS; ++n) ring.fetch(n, row + n * stride, rows);
  F2 wh[kHold ? NV : 1][U], bh[kHold ? NV : 1][U];
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (R::in(lane, i, W)) {
        load_w<V>(w, R::column(lane, i), 1.0f, wh[i]);
        load_w<V>(b, R::column(lane, i), 0.0f, bh[i]);
      }
    }
  }
  int half = 0;
  for (int n = 0; row < rows; row += stride, n = n + 1 < SLOTS ? n + 1 : 0) {   // whole warps, or the whole CTA
    const int64_t base = row * W;
    ring.wait();
    F2 v[NV][U];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < U; ++e) v[i][e] = splat(0.f);
      if (R::in(lane, i, W)) {
        ring.get(n, 0, i, row).unpack(v[i]);
        if (RES) {
          F2 u[U];
          ring.get(n, RES ? 1 : 0, i, row).unpack(u);
#pragma unroll
          for (int e = 0; e < U; ++e) v[i][e] = add2(v[i][e], u[e]);
        }
      }
    }
    ring.fetch(n, row + SLOTS * stride, rows);
    if (sum_out) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (R::in(lane, i, W)) store_pack<T, V>(sum_out + base + R::column(lane, i), v[i]);
    }
    float m[2];   // the deviations' sum and that of their squares
    center<R>(v, W, lane, red, half, m[0], m[1]);
    row_sums<R::G>(m, red, half);
    const float shift = m[0] * inv_w, rf = inverse_std(m[1], shift, inv_w, eps);
    const F2 r = splat(rf), r0 = splat(-shift * rf);   // z = (dev - shift) r
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (R::in(lane, i, W)) {
        F2 wv[U], bv[U];
        if constexpr (!kHold) {
          load_w<V>(w, R::column(lane, i), 1.0f, wv);
          load_w<V>(b, R::column(lane, i), 0.0f, bv);
        }
#pragma unroll
        for (int e = 0; e < U; ++e)
          v[i][e] = fma2(fma2(v[i][e], r, r0), kHold ? wh[kHold ? i : 0][e] : wv[e], kHold ? bh[kHold ? i : 0][e] : bv[e]);
        store_pack<T, V>(out + base + R::column(lane, i), v[i]);
      }
    }
  }
}

// As the forward; a thread keeps the sums of dout z and dout over its rows for its own columns, and
// the CTA's go to partial[blockIdx.x] as [dw: W][db: W].
template <class R, int TPB, bool SUM, int SLOTS, int BLOCKS>
__global__ void __launch_bounds__(TPB, BLOCKS)
layer_norm_backward_kernel(const typename R::T* s, const typename R::T* dout, const typename R::T* dsum,
                           const float* __restrict__ w, typename R::T* dx, float* __restrict__ partial, int rows, int W,
                           float eps) {
  using T = typename R::T;
  constexpr int V = R::V, NV = R::NV, U = R::U;
  constexpr bool kHold = NV * V <= 16;
  __shared__ Sums red;
  extern __shared__ __align__(16) unsigned char ring_smem[];
  const int lane = threadIdx.x % R::G, group = threadIdx.x / R::G;
  const float inv_w = 1.0f / static_cast<float>(W);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (TPB / R::G);
  int64_t row = static_cast<int64_t>(blockIdx.x) * (TPB / R::G) + group;
  Ring<R, TPB, SUM ? 3 : 2, SLOTS> ring;
  ring.base = reinterpret_cast<Pack<T, V>*>(ring_smem);
  ring.src[0] = s;
  ring.src[1] = dout;
  if (SUM) ring.src[SUM ? 2 : 0] = dsum;
  ring.W = W;
  ring.lane = lane;
#pragma unroll
  for (int n = 0; n < SLOTS; ++n) ring.fetch(n, row + n * stride, rows);
  int half = 0;
  F2 dw[NV][U], db[NV][U], wh[kHold ? NV : 1][U];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < U; ++e) dw[i][e] = db[i][e] = splat(0.f);
    if constexpr (kHold) {
      if (R::in(lane, i, W)) load_w<V>(w, R::column(lane, i), 1.0f, wh[kHold ? i : 0]);
    }
  }
  for (int n = 0; row < rows; row += stride, n = n + 1 < SLOTS ? n + 1 : 0) {
    const int64_t base = row * W;
    ring.wait();
    F2 v[NV][U], d[NV][U];
    Pack<T, V> u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < U; ++e) v[i][e] = d[i][e] = splat(0.f);
      if (R::in(lane, i, W)) {
        ring.get(n, 0, i, row).unpack(v[i]);
        ring.get(n, 1, i, row).unpack(d[i]);
        if (SUM) u[i] = ring.get(n, SUM ? 2 : 0, i, row);
      }
    }
    ring.fetch(n, row + SLOTS * stride, rows);
    // One reduction for the deviations' sum, that of their squares, and the two of g: z = (dev - shift) r, so the sum of
    // g z is r times that of g dev less shift times that of g.
    float m[4];
    center<R>(v, W, lane, red, half, m[0], m[1]);
    F2 sg = splat(0.f), sgd = splat(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (R::in(lane, i, W)) {
        F2 wv[U];
        if constexpr (!kHold) load_w<V>(w, R::column(lane, i), 1.0f, wv);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const F2 g = mul2(d[i][e], kHold ? wh[kHold ? i : 0][e] : wv[e]);
          sg = add2(sg, g);
          sgd = fma2(g, v[i][e], sgd);
        }
      }
    }
    m[2] = both(sg);
    m[3] = both(sgd);
    row_sums<R::G>(m, red, half);
    const float shift = m[0] * inv_w, r = inverse_std(m[1], shift, inv_w, eps);
    const F2 mg = splat(-m[2] * inv_w), mgz = splat(-fmaf(-shift, m[2], m[3]) * r * inv_w);
    const F2 r2 = splat(r), r0 = splat(-shift * r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (R::in(lane, i, W)) {
        F2 o[U], wv[U];
        if constexpr (!kHold) load_w<V>(w, R::column(lane, i), 1.0f, wv);
#pragma unroll
        for (int e = 0; e < U; ++e) o[e] = splat(0.f);
        if (SUM) u[i].unpack(o);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const F2 z = fma2(v[i][e], r2, r0);
          dw[i][e] = fma2(d[i][e], z, dw[i][e]);
          db[i][e] = add2(db[i][e], d[i][e]);
          const F2 g = fma2(d[i][e], kHold ? wh[kHold ? i : 0][e] : wv[e], mg);
          o[e] = fma2(r2, fma2(z, mgz, g), o[e]);
        }
        store_pack<T, V>(dx + base + R::column(lane, i), o);
      }
    }
  }
  if (!partial) return;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * W;
  auto put = [&](float* to, bool add) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = R::column(lane, i) + e;
        if (c < W) {
          const float2 a = split(dw[i][e / 2]), b = split(db[i][e / 2]);
          to[c] = (add ? to[c] : 0.f) + (e % 2 ? a.y : a.x);
          to[W + c] = (add ? to[W + c] : 0.f) + (e % 2 ? b.y : b.x);
        }
      }
    }
  };
  if constexpr (R::G == TPB) {
    put(out, false);
  } else {   // the CTA's rows-in-parallel, one after the other
    float* fold = reinterpret_cast<float*>(ring_smem);   // [2][W]; nothing is on its way any more
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (int k = 0; k < TPB / R::G; ++k) {
      __syncthreads();
      if (group == k) put(fold, k > 0);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * W; c += TPB) out[c] = fold[c];
  }
}

// dw[c] and db[c]: the CTAs' partial sums, added in a fixed order: 32 threads a column, each over
// every 32nd CTA, then the 32 in turn.
__global__ void __launch_bounds__(1024) layer_norm_weight_sum_kernel(const float* __restrict__ partial, int parts,
                                                                     int W, float* __restrict__ dw,
                                                                     float* __restrict__ db) {
  __shared__ float red[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;   // column of [dw: W][db: W]
  float a = 0.f;
  if (c < 2 * W) {
#pragma unroll 8
    for (int k = ty; k < parts; k += 32) a += __ldg(partial + static_cast<int64_t>(k) * 2 * W + c);
  }
  red[ty][tx] = a;
  __syncthreads();
  if (ty == 0 && c < 2 * W) {
#pragma unroll
    for (int k = 1; k < 32; ++k) a += red[k][tx];
    if (c < W) {
      if (dw) dw[c] = a;
    } else if (db) {
      db[c - W] = a;
    }
  }
}

struct LnArgs {
  const void *x, *residual, *dout, *dsum;
  const float *w, *b;
  void *out, *sum_out;
  float *partial, *dw, *db;
  int rows, W;
  float eps;
  cudaStream_t stream;
};

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  return n;
}
// CTAs: one for each TPB / G rows, no more than fit at once.
unsigned ln_grid(int rows, int per, int blocks) {
  const int64_t need = (static_cast<int64_t>(rows) + per - 1) / per, fit = static_cast<int64_t>(blocks) * sm_count();
  return static_cast<unsigned>(need < fit ? need : fit);
}
constexpr int clamp_slots(int n) { return n < 1 ? 1 : n > 4 ? 4 : n; }

template <class R, bool RES> cudaError_t ln_forward(const LnArgs& a) {
  using T = typename R::T;
  constexpr int G = R::G, TPB = G == 32 ? 128 : G;
  // wide rows: CTAs that stay, 512 threads an SM, their shared memory full of rows to come; narrow ones: a row
  // a group, as many as fit (65536 x 1024 bf16: 93 us against 105 from shared memory; fp32 65537 x 768: 122
  // against 149)
  constexpr bool kStay = R::V > 1 && G >= 256;
  constexpr int BLOCKS = kStay ? (512 / TPB > 0 ? 512 / TPB : 1) : 1;
  constexpr int SLOTS = kStay ? clamp_slots(200 * 1024 / (BLOCKS * TPB) / 16 / ((RES ? 2 : 1) * R::NV)) : 0;
  constexpr size_t smem = Ring<R, TPB, RES ? 2 : 1, SLOTS>::kBytes;
  auto kernel = layer_norm_kernel<R, TPB, RES, SLOTS, BLOCKS>;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int per = TPB / G;
  const unsigned grid = kStay ? ln_grid(a.rows, per, BLOCKS) : static_cast<unsigned>((a.rows - 1) / per + 1);
  kernel<<<grid, TPB, smem, a.stream>>>(static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.w, a.b,
                                        static_cast<T*>(a.out), static_cast<T*>(a.sum_out), a.rows, a.W, a.eps);
  return cudaGetLastError();
}
// The backward's CTAs: as many threads an SM as the sums' registers allow, in no more than 8 CTAs. Each has a part of the
// sums to write and to be added, and more of them cost more than their threads gain: of 64 threads, 8 against 10
// (fp32) or 16: 65536 x 600 fp32 115 us against 122, 131072 x 512 bf16 94 against 101, 3000 x 512 17 against 25 (only rows read
// element by element gain: 100000 x 129 107 against 77).
template <int V, int NV, int G> struct Back {
  static constexpr int TPB = G == 32 ? 256 : G, per = TPB / G;
  static constexpr int THREADS = NV * V <= 8 ? 1024 : 512;   // NV * V values of a row, and of each sum, in a thread
  static constexpr int FIT = THREADS / TPB, BLOCKS = FIT < 1 ? 1 : FIT > 8 ? 8 : FIT;
};
template <class R, bool SUM> cudaError_t ln_backward(const LnArgs& a) {
  using T = typename R::T;
  using S = Back<R::V, R::NV, R::G>;
  constexpr int TPB = S::TPB, per = S::per, BLOCKS = S::BLOCKS;
  constexpr int SLOTS = R::V == 1 ? 0 : clamp_slots(200 * 1024 / (BLOCKS * TPB) / 16 / ((SUM ? 3 : 2) * R::NV));
  constexpr size_t ring = Ring<R, TPB, SUM ? 3 : 2, SLOTS>::kBytes;
  const size_t fold = per == 1 ? 0 : 2 * sizeof(float) * a.W, smem = ring > fold ? ring : fold;
  auto kernel = layer_norm_backward_kernel<R, TPB, SUM, SLOTS, BLOCKS>;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = ln_grid(a.rows, per, BLOCKS);
  kernel<<<grid, TPB, smem, a.stream>>>(static_cast<const T*>(a.x), static_cast<const T*>(a.dout),
                                        static_cast<const T*>(a.dsum), a.w, static_cast<T*>(a.out), a.partial, a.rows,
                                        a.W, a.eps);
  if (a.partial)
    layer_norm_weight_sum_kernel<<<(2 * a.W + 31) / 32, 1024, 0, a.stream>>>(a.partial, static_cast<int>(grid), a.W, a.dw,
                                                                            a.db);
  return cudaGetLastError();
}

// The threads that share a row and how much of it each holds, by the row's vectors.  The backward's sums
// take registers, so its rows have more threads with less each (8192 wide: 512 threads of two vectors 117
// us, 1024 of one 144; 65536 x 1024: 128 threads of one vector 114 us, a warp of four 215).  Rows of 129 to 192 vectors lie
// in 64 threads of three, not in 128 of two: fp32 65536 x 520 61 us against 91, its backward 81 against 116, 65537 x 768 70
// against 95 and 114 against 124, bf16 32768 x 1280 48 against 66; but the bf16 backward in 128 (32768 x 1280: 76
// us against 92, 32768 x 1536 82 against 92).
template <typename T, int V, int NV, int G> cudaError_t ln_fwd(const LnArgs& a) {
  if (V > 1 && a.W == V * NV * G)
    return a.residual ? ln_forward<Row<T, V, NV, G, V != 1>, true>(a) : ln_forward<Row<T, V, NV, G, V != 1>, false>(a);
  return a.residual ? ln_forward<Row<T, V, NV, G, false>, true>(a) : ln_forward<Row<T, V, NV, G, false>, false>(a);
}
template <typename T, int V, int NV, int G> cudaError_t ln_bwd(const LnArgs& a) {
  if (V > 1 && a.W == V * NV * G)
    return a.dsum ? ln_backward<Row<T, V, NV, G, V != 1>, true>(a) : ln_backward<Row<T, V, NV, G, V != 1>, false>(a);
  return a.dsum ? ln_backward<Row<T, V, NV, G, false>, true>(a) : ln_backward<Row<T, V, NV, G, false>, false>(a);
}
template <int NV_, int G_> struct Band {
  static constexpr int NV = NV_, G = G_;
};
template <int V, class F> auto forward_band(int W, F f) {
  const int vecs = (W + V - 1) / V;
  if (vecs <= 32) return f(Band<1, 32>{});
  if (vecs <= 64) return f(Band<2, 32>{});
  if (vecs <= 128) return f(Band<4, 32>{});
  if (vecs <= 192) return f(Band<3, 64>{});
  if (vecs <= 256) return f(Band<2, 128>{});
  if (vecs <= 512) return f(Band<2, 256>{});
  if (vecs <= 1024) return f(Band<2, 512>{});
  if constexpr (V == 8) return f(Band<4, 512>{});
  if (vecs <= 2048) return f(Band<4, 512>{});
  if constexpr (V == 4) return f(Band<4, 1024>{});
  if (vecs <= 4096) return f(Band<4, 1024>{});
  return f(Band<16, 1024>{});
}
template <int V, class F> auto backward_band(int W, F f) {
  const int vecs = (W + V - 1) / V;
  if (vecs <= 32) return f(Band<1, 32>{});
  if (vecs <= 64) return f(Band<1, 64>{});
  if (vecs <= 128) return f(Band<1, 128>{});
  if (vecs <= 192 && V < 8) return f(Band<3, 64>{});   // of 8 values they and both their sums are 72 registers
  if (vecs <= 256) return f(Band<2, 128>{});
  if (vecs <= 512) return f(Band<2, 256>{});
  if (vecs <= 1024) return f(Band<2, 512>{});
  if constexpr (V == 8) return f(Band<4, 512>{});
  if (vecs <= 2048) return f(Band<4, 512>{});
  if constexpr (V == 4) return f(Band<4, 1024>{});
  if (vecs <= 4096) return f(Band<4, 1024>{});
  return f(Band<16, 1024>{});
}
static_assert(kMaxNormWidth <= 16384, "the widest band");
template <typename T, int V> cudaError_t ln_launch(const LnArgs& a, bool backward) {
  if (backward)
    return backward_band<V>(a.W, [&](auto b) { return ln_bwd<T, V, decltype(b)::NV, decltype(b)::G>(a); });
  return forward_band<V>(a.W, [&](auto b) { return ln_fwd<T, V, decltype(b)::NV, decltype(b)::G>(a); });
}
// How many parts of the sums the backward's CTAs write: what its grid is, and its workspace.
template <int V> size_t ln_parts(int rows, int W) {
  return backward_band<V>(W, [&](auto b) -> size_t {
    using S = Back<V, decltype(b)::NV, decltype(b)::G>;
    return ln_grid(rows, S::per, S::BLOCKS);
  });
}

cudaError_t launch_layer_norm(const LnArgs& a, la_dtype dt, bool backward) {
  if (dt == LA_BF16) return a.W % 8 == 0 ? ln_launch<uint16_t, 8>(a, backward) : ln_launch<uint16_t, 1>(a, backward);
  return a.W % 4 == 0 ? ln_launch<float, 4>(a, backward) : ln_launch<float, 1>(a, backward);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Of either type.
size_t ln_ws_bytes(int rows, int W) {
  const size_t bf16 = W % 8 == 0 ? ln_parts<8>(rows, W) : ln_parts<1>(rows, W);
  const size_t f32 = W % 4 == 0 ? ln_parts<4>(rows, W) : ln_parts<1>(rows, W);
  const size_t n = sizeof(float) * 2 * W * (bf16 > f32 ? bf16 : f32);
  return n < 256 ? 256 : (n + 255) & ~size_t(255);
}

size_t ln_bytes(int rows, int W, la_dtype dt) { return static_cast<size_t>(rows) * W * (dt == LA_BF16 ? 2 : 4); }

bool ln_valid(int rows, int W, la_dtype dt, float eps, const float* w, const float* b) {
  return rows >= 0 && W >= 1 && (dt == LA_F32 || dt == LA_BF16) && eps > 0.0f && (!w || aligned16(w)) &&
         (!b || aligned16(b));
}

}  // namespace
}  // namespace la

extern "C" {

la_status lightning_attn_layer_norm(const void* x, const void* residual, const float* weight, const float* bias,
                                    void* out, void* sum_out, int rows, int W, la_dtype dtype, float eps,
                                    la_stream_t stream) {
  if (!la::ln_valid(rows, W, dtype, eps, weight, bias)) return LA_ERR_INVALID_ARG;
  if (W > la::kMaxNormWidth) return LA_ERR_UNSUPPORTED;
  if (rows == 0) return LA_OK;
  if (!x || !out || !la::aligned16(x) || !la::aligned16(out) || (residual && !la::aligned16(residual)) ||
      (sum_out && !la::aligned16(sum_out)))
    return LA_ERR_INVALID_ARG;
  // rows are written while others are still to be read: in place or apart, nothing between
  const size_t n = la::ln_bytes(rows, W, dtype), nw = sizeof(float) * W;
  if (la::overlap(out, n, sum_out, n)) return LA_ERR_INVALID_ARG;
  for (const void* to : {static_cast<const void*>(out), static_cast<const void*>(sum_out)})
    if (la::shifted(to, n, x, n) || la::shifted(to, n, residual, n) || la::overlap(to, n, weight, nw) ||
        la::overlap(to, n, bias, nw))
      return LA_ERR_INVALID_ARG;
  la::LnArgs a{};
  a.x = x; a.residual = residual; a.w = weight; a.b = bias; a.out = out; a.sum_out = sum_out;
  a.rows = rows; a.W = W; a.eps = eps; a.stream = reinterpret_cast<cudaStream_t>(stream);
  return la::launch_layer_norm(a, dtype, false) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status lightning_attn_layer_norm_backward(const void* s, const void* dout, const void* dsum, const float* weight,
                                             void* dx, float* dweight, float* dbias, int rows, int W, la_dtype dtype,
                                             float eps, void* workspace, size_t workspace_bytes, la_stream_t stream) {
  if (!la::ln_valid(rows, W, dtype, eps, weight, nullptr)) return LA_ERR_INVALID_ARG;
  if (W > la::kMaxNormWidth) return LA_ERR_UNSUPPORTED;
  const size_t nw = sizeof(float) * W;
  if ((dweight && !la::aligned16(dweight)) || (dbias && !la::aligned16(dbias)) || la::overlap(dweight, nw, dbias, nw))
    return LA_ERR_INVALID_ARG;
  const bool sums = dweight || dbias;
  if (sums && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
               workspace_bytes < la::ln_ws_bytes(rows, W)))
    return LA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {
    for (float* p : {dweight, dbias})
      if (p && cudaMemsetAsync(p, 0, sizeof(float) * W, st) != cudaSuccess) return LA_ERR_CUDA;
    return LA_OK;
  }
  if (!s || !dout || !dx || !la::aligned16(s) || !la::aligned16(dout) || !la::aligned16(dx) ||
      (dsum && !la::aligned16(dsum)))
    return LA_ERR_INVALID_ARG;
  const size_t n = la::ln_bytes(rows, W, dtype), parts = sums ? la::ln_ws_bytes(rows, W) : 0;
  if (la::shifted(dx, n, s, n) || la::shifted(dx, n, dout, n) || la::shifted(dx, n, dsum, n) ||
      la::overlap(dx, n, weight, nw) || la::overlap(dx, n, dweight, nw) || la::overlap(dx, n, dbias, nw))
    return LA_ERR_INVALID_ARG;
  for (const void* t : {s, dout, dsum, static_cast<const void*>(dx)})
    if (la::overlap(workspace, parts, t, n)) return LA_ERR_INVALID_ARG;
  for (const void* t : {weight, static_cast<const float*>(dweight), static_cast<const float*>(dbias)})
    if (la::overlap(workspace, parts, t, nw)) return LA_ERR_INVALID_ARG;
  la::LnArgs a{};
  a.x = s; a.dout = dout; a.dsum = dsum; a.w = weight; a.out = dx; a.dw = dweight; a.db = dbias;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  a.rows = rows; a.W = W; a.eps = eps; a.stream = st;
  return la::launch_layer_norm(a, dtype, true) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

size_t lightning_attn_layer_norm_workspace_size(int rows, int W) {
  if (rows < 0 || W < 1 || W > la::kMaxNormWidth) return 0;
  return la::ln_ws_bytes(rows, W);
}

}  // extern "C"
