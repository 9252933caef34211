// Layer norm over rows of W values with the residual addition in front of it, forward and
// backward (sm_100a).
//
//   s = x + residual,  z = (s - mean) r,  r = 1 / sqrt(mean((s - mean)^2) + eps),  y = z w + b
//   g = dout w,  dx = r (g - mean(g) - z mean(g z)) + dsum,  dw = sum dout z,  db = sum dout
//
// A row stays in the registers of the G threads that share it (a warp, or a CTA) between its
// one read and its one write, so the deviations are squared after the mean is known and both
// passes touch memory once.
#include "la_common.cuh"

namespace la {
namespace {

// One thread's V consecutive values, as loaded (16 bytes, or one element).
template <typename T, int V> struct Pack;
template <> struct Pack<uint16_t, 8> {
  uint4 r;
  __device__ __forceinline__ void unpack(float* o) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void pack(const float* o) {
    r = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
  }
};
template <> struct Pack<float, 4> {
  float4 r;
  __device__ __forceinline__ void unpack(float* o) const { o[0] = r.x; o[1] = r.y; o[2] = r.z; o[3] = r.w; }
  __device__ __forceinline__ void pack(const float* o) { r = make_float4(o[0], o[1], o[2], o[3]); }
};
template <> struct Pack<uint16_t, 1> {
  uint16_t r;
  __device__ __forceinline__ void unpack(float* o) const { o[0] = bf16_bits_to_f32(r); }
  __device__ __forceinline__ void pack(const float* o) { r = f32_to_bf16_bits(o[0]); }
};
template <> struct Pack<float, 1> {
  float r;
  __device__ __forceinline__ void unpack(float* o) const { o[0] = r; }
  __device__ __forceinline__ void pack(const float* o) { r = o[0]; }
};

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V> __device__ __forceinline__ void store_pack(T* p, const float* o) {
  Pack<T, V> k;
  k.pack(o);
  *reinterpret_cast<Pack<T, V>*>(p) = k;
}
// V fp32 values of the weight or bias (`fill` where there is none).
template <int V> __device__ __forceinline__ void load_w(const float* p, int c, float fill, float* o) {
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = fill;
  if (!p) return;
  if constexpr (V == 1) {
    o[0] = __ldg(p + c);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(p + c + i));
      o[i] = t.x; o[i + 1] = t.y; o[i + 2] = t.z; o[i + 3] = t.w;
    }
  }
}

// Sum of two values over the G threads of a row, in every one of them, in a fixed order.
// `red` alternates between calls, so one barrier a call is enough.
template <int G> __device__ __forceinline__ float2 row_sum(float a, float b, float2 (*red)[32], int& half) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (G == 32) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) red[half][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  a = 0.f;
  b = 0.f;
#pragma unroll
  for (int i = 0; i < G / 32; ++i) {
    a += red[half][i].x;
    b += red[half][i].y;
  }
  half ^= 1;
  return make_float2(a, b);
}

// Mean and 1 / sqrt(variance + eps) of a row held in registers; v becomes v - mean.
template <int V, int NV, int G>
__device__ __forceinline__ float center(float (*v)[V], int W, float eps, int lane, float2 (*red)[32],
                                        int& half) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) a += v[i][e];
  // divided, not multiplied by 1 / W: the mean of equal values is then that value
  const float mean = row_sum<G>(a, 0.f, red, half).x / static_cast<float>(W);
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = (lane + i * G) * V < W;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[i][e] = in ? v[i][e] - mean : 0.f;
      q = fmaf(v[i][e], v[i][e], q);
    }
  }
  return 1.0f / sqrtf(row_sum<G>(q, 0.f, red, half).x / static_cast<float>(W) + eps);
}

template <typename T, int V, int NV, int G, int TPB>
__global__ void __launch_bounds__(TPB) layer_norm_kernel(const T* x, const T* residual, const float* __restrict__ w,
                                                         const float* __restrict__ b, T* out, T* sum_out, int rows,
                                                         int W, float eps) {
  __shared__ float2 red[2][32];
  const int lane = threadIdx.x % G;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (TPB / G) + threadIdx.x / G;
  if (row >= rows) return;   // whole warps (G == 32), or no one (G == TPB)
  int half = 0;
  const int64_t base = row * W;
  float v[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * G) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] = 0.f;
    if (c < W) load_pack<T, V>(x + base + c).unpack(v[i]);
  }
  if (residual) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
      if (c < W) {
        float u[V];
        load_pack<T, V>(residual + base + c).unpack(u);
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] += u[e];
      }
    }
  }
  if (sum_out) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
      if (c < W) store_pack<T, V>(sum_out + base + c, v[i]);
    }
  }
  const float r = center<V, NV, G>(v, W, eps, lane, red, half);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * G) * V;
    if (c < W) {
      float wv[V], bv[V];
      load_w<V>(w, c, 1.0f, wv);
      load_w<V>(b, c, 0.0f, bv);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = fmaf(v[i][e] * r, wv[e], bv[e]);
      store_pack<T, V>(out + base + c, v[i]);
    }
  }
}

// The CTA's rows are blockIdx.x * (TPB / G) + threadIdx.x / G, then every gridDim.x * (TPB / G)
// further.  A thread keeps the sums of dout z and dout over its rows for its own columns;
// the CTA's sums go to partial[blockIdx.x] as [dw: W][db: W].
template <typename T, int V, int NV, int G, int TPB>
__global__ void __launch_bounds__(TPB) layer_norm_backward_kernel(const T* s, const T* dout, const T* dsum,
                                                                  const float* __restrict__ w, T* dx,
                                                                  float* __restrict__ partial, int rows, int W,
                                                                  float eps) {
  __shared__ float2 red[2][32];
  extern __shared__ float fold[];   // G == 32 with partial: [2][W]
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const float inv_w = 1.0f / static_cast<float>(W);
  int half = 0;
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.f;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (TPB / G) + group; row < rows;
       row += static_cast<int64_t>(gridDim.x) * (TPB / G)) {
    const int64_t base = row * W;
    float v[NV][V], d[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = d[i][e] = 0.f;
      if (c < W) {
        load_pack<T, V>(s + base + c).unpack(v[i]);
        load_pack<T, V>(dout + base + c).unpack(d[i]);
      }
    }
    const float r = center<V, NV, G>(v, W, eps, lane, red, half);
    float sg = 0.f, sgz = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
      if (c < W) {
        float wv[V];
        load_w<V>(w, c, 1.0f, wv);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float z = v[i][e] * r;
          dw[i][e] = fmaf(d[i][e], z, dw[i][e]);
          db[i][e] += d[i][e];
          v[i][e] = z;
          d[i][e] *= wv[e];
          sg += d[i][e];
          sgz = fmaf(d[i][e], z, sgz);
        }
      }
    }
    const float2 m = row_sum<G>(sg, sgz, red, half);
    const float mg = m.x * inv_w, mgz = m.y * inv_w;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * G) * V;
      if (c < W) {
        float u[V];
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = 0.f;
        if (dsum) load_pack<T, V>(dsum + base + c).unpack(u);
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] += r * (d[i][e] - mg - v[i][e] * mgz);
        store_pack<T, V>(dx + base + c, u);
      }
    }
  }
  if (!partial) return;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * W;
  for (int k = 0; k < TPB / G; ++k) {   // the CTA's rows-in-parallel, one after the other
    if (group == k) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int c = (lane + i * G) * V + e;
          if (c < W) {
            if (G == TPB) {
              out[c] = dw[i][e];
              out[W + c] = db[i][e];
            } else {
              fold[c] = k ? fold[c] + dw[i][e] : dw[i][e];
              fold[W + c] = k ? fold[W + c] + db[i][e] : db[i][e];
            }
          }
        }
      }
    }
    if (G != TPB) __syncthreads();
  }
  if (G != TPB)
    for (int c = threadIdx.x; c < 2 * W; c += TPB) out[c] = fold[c];
}

// dw[c] and db[c]: the CTAs' partial sums, added in a fixed order: 8 threads a column, each
// over every 8th CTA, then the 8 in turn.
__global__ void __launch_bounds__(256) layer_norm_weight_sum_kernel(const float* __restrict__ partial, int parts,
                                                                    int W, float* __restrict__ dw,
                                                                    float* __restrict__ db) {
  __shared__ float red[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;   // column of [dw: W][db: W]
  float a = 0.f;
  if (c < 2 * W)
    for (int k = ty; k < parts; k += 8) a += partial[static_cast<int64_t>(k) * 2 * W + c];
  red[ty][tx] = a;
  __syncthreads();
  if (ty == 0 && c < 2 * W) {
#pragma unroll
    for (int k = 1; k < 8; ++k) a += red[k][tx];
    if (c < W) {
      if (dw) dw[c] = a;
    } else if (db) {
      db[c - W] = a;
    }
  }
}

constexpr int kMaxParts = 592;   // CTAs of the backward pass: 4 for each of 148 SMs

struct LnArgs {
  const void *x, *residual, *dout, *dsum;
  const float *w, *b;
  void *out, *sum_out;
  float *partial, *dw, *db;
  int rows, W;
  float eps;
  cudaStream_t stream;
};

template <typename T, int V, int NV, int G> cudaError_t ln_forward(const LnArgs& a) {
  constexpr int TPB = G == 32 ? 128 : G;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.rows) + TPB / G - 1) / (TPB / G));
  layer_norm_kernel<T, V, NV, G, TPB><<<grid, TPB, 0, a.stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.w, a.b, static_cast<T*>(a.out),
      static_cast<T*>(a.sum_out), a.rows, a.W, a.eps);
  return cudaGetLastError();
}
template <typename T, int V, int NV, int G> cudaError_t ln_backward(const LnArgs& a) {
  constexpr int TPB = G == 32 ? 256 : G;
  const int64_t need = (static_cast<int64_t>(a.rows) + TPB / G - 1) / (TPB / G);
  const int grid = static_cast<int>(need < kMaxParts ? need : kMaxParts);
  const size_t smem = G == TPB || !a.partial ? 0 : 2 * sizeof(float) * a.W;
  layer_norm_backward_kernel<T, V, NV, G, TPB><<<grid, TPB, smem, a.stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.dout), static_cast<const T*>(a.dsum), a.w,
      static_cast<T*>(a.out), a.partial, a.rows, a.W, a.eps);
  if (a.partial)
    layer_norm_weight_sum_kernel<<<(2 * a.W + 31) / 32, 256, 0, a.stream>>>(a.partial, grid, a.W, a.dw, a.db);
  return cudaGetLastError();
}

// The threads that share a row and how much of it each holds, by the row's vectors.
template <typename T, int V> cudaError_t ln_launch(const LnArgs& a, bool backward) {
  const int vecs = (a.W + V - 1) / V;
#define LA_LN(NV, G) return backward ? ln_backward<T, V, NV, G>(a) : ln_forward<T, V, NV, G>(a)
  if (vecs <= 32) LA_LN(1, 32);
  if (vecs <= 64) LA_LN(2, 32);
  if (vecs <= 128) LA_LN(4, 32);
  if (vecs <= 256) LA_LN(2, 128);
  if (vecs <= 512) LA_LN(2, 256);
  if (vecs <= 1024) LA_LN(2, 512);
  if (vecs <= 2048) LA_LN(4, 512);
  if (vecs <= 4096) LA_LN(4, 1024);
  if (V == 1) LA_LN(16, 1024);
#undef LA_LN
  return cudaErrorInvalidValue;
}

cudaError_t launch_layer_norm(const LnArgs& a, la_dtype dt, bool backward) {
  if (dt == LA_BF16) return a.W % 8 == 0 ? ln_launch<uint16_t, 8>(a, backward) : ln_launch<uint16_t, 1>(a, backward);
  return a.W % 4 == 0 ? ln_launch<float, 4>(a, backward) : ln_launch<float, 1>(a, backward);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t ln_ws_bytes(int rows, int W) {
  const size_t parts = static_cast<size_t>(rows < kMaxParts ? rows : kMaxParts);
  const size_t n = sizeof(float) * 2 * W * parts;
  return n < 256 ? 256 : (n + 255) & ~size_t(255);
}

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
      (sum_out && (!la::aligned16(sum_out) || sum_out == out)))
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
  if ((dweight && !la::aligned16(dweight)) || (dbias && !la::aligned16(dbias)) || (dweight && dweight == dbias))
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
