// Gated linear recurrence h_t = a_t h_{t-1} + b_t, a = sigmoid(f), b = x or (1 - a) x, channel
// by channel: forward, one-token step and backward (sm_100a).
//
// One thread owns one channel of one sequence and walks the time axis.
#include "la_common.cuh"

namespace la {

void set_last_path(const char* path);

namespace {

constexpr int kCkRows = LA_RECURRENCE_CHECKPOINT_ROWS;

struct RecArgs {
  const void *x, *f, *dout;
  void *out, *dx, *df;
  const float *s0, *ds1;
  float *s1, *ds0, *ck;
  const int* cu;
  int nseq, T, W, tied;
  int64_t tokens;
  ErrRec* err;
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

// Rows of sequence s; a malformed one has none (and is reported).
__device__ __forceinline__ void seq_rows(const RecArgs& p, int s, int64_t& lo, int64_t& hi) {
  if (!p.cu) {
    lo = static_cast<int64_t>(s) * p.T;
    hi = lo + p.T;
    return;
  }
  lo = __ldg(p.cu + s);
  hi = __ldg(p.cu + s + 1);
  if (lo < 0 || hi < lo || hi > p.tokens) {
    report(p.err, LA_ERR_DEVICE, SITE_VARLEN_CU, static_cast<unsigned>(s), 0);
    lo = hi = 0;
  }
}

template <typename T>
__global__ void __launch_bounds__(128) rec_forward_kernel(RecArgs p) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.W) return;
  const T* x = static_cast<const T*>(p.x);
  const T* f = static_cast<const T*>(p.f);
  T* out = static_cast<T*>(p.out);
  for (int s = blockIdx.y; s < p.nseq; s += gridDim.y) {
    int64_t lo, hi;
    seq_rows(p, s, lo, hi);
    const int64_t si = static_cast<int64_t>(s) * p.W + c;
    float h = p.s0 ? p.s0[si] : 0.f;
    for (int64_t t = lo; t < hi; ++t) {
      if (p.ck && t % kCkRows == 0) p.ck[t / kCkRows * p.W + c] = h;
      const float xv = load_elem<T>(x, t * p.W + c);
      const Gate g = gate_of(load_elem<T>(f, t * p.W + c));
      h = fmaf(g.a, h, p.tied ? g.keep * xv : xv);
      if (out) store_elem<T>(out, t * p.W + c, h);
    }
    if (p.s1) p.s1[si] = h;
  }
}

template <typename T>
__global__ void __launch_bounds__(128) rec_backward_kernel(RecArgs p) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.W) return;
  const T* x = static_cast<const T*>(p.x);
  const T* f = static_cast<const T*>(p.f);
  const T* dout = static_cast<const T*>(p.dout);
  T* dx = static_cast<T*>(p.dx);
  T* df = static_cast<T*>(p.df);
  for (int s = blockIdx.y; s < p.nseq; s += gridDim.y) {
    int64_t lo, hi;
    seq_rows(p, s, lo, hi);
    const int64_t si = static_cast<int64_t>(s) * p.W + c;
    float carry = p.ds1 ? p.ds1[si] : 0.f;   // what flows back into the state after row t
    float prev[kCkRows];
    for (int64_t end = hi; end > lo;) {      // blocks between checkpoints, last first
      int64_t begin = (end - 1) / kCkRows * kCkRows;
      float h;
      if (begin > lo) {
        h = p.ck[begin / kCkRows * p.W + c];
      } else {
        begin = lo;
        h = p.s0 ? p.s0[si] : 0.f;
      }
      for (int64_t t = begin; t < end; ++t) {
        prev[t - begin] = h;
        const float xv = load_elem<T>(x, t * p.W + c);
        const Gate g = gate_of(load_elem<T>(f, t * p.W + c));
        h = fmaf(g.a, h, p.tied ? g.keep * xv : xv);
      }
      for (int64_t t = end - 1; t >= begin; --t) {
        const float xv = load_elem<T>(x, t * p.W + c);
        const Gate g = gate_of(load_elem<T>(f, t * p.W + c));
        const float G = load_elem<T>(dout, t * p.W + c) + carry;
        store_elem<T>(dx, t * p.W + c, p.tied ? g.keep * G : G);
        store_elem<T>(df, t * p.W + c, G * g.a * g.keep * (p.tied ? prev[t - begin] - xv : prev[t - begin]));
        carry = g.a * G;
      }
      end = begin;
    }
    if (p.ds0) p.ds0[si] = carry;
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

dim3 rec_grid(const RecArgs& p) {
  return dim3(static_cast<unsigned>((p.W + 127) / 128), static_cast<unsigned>(p.nseq < 65535 ? p.nseq : 65535));
}

cudaError_t launch_rec_forward(const RecArgs& p, la_dtype dt, cudaStream_t stream) {
  if (dt == LA_BF16) rec_forward_kernel<uint16_t><<<rec_grid(p), 128, 0, stream>>>(p);
  else rec_forward_kernel<float><<<rec_grid(p), 128, 0, stream>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_rec_backward(const RecArgs& p, la_dtype dt, cudaStream_t stream) {
  if (dt == LA_BF16) rec_backward_kernel<uint16_t><<<rec_grid(p), 128, 0, stream>>>(p);
  else rec_backward_kernel<float><<<rec_grid(p), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace: [error record] [backward: checkpoints, for a call that was given none].
size_t checkpoint_bytes(int64_t tokens, int W) {
  return up256(sizeof(float) * static_cast<size_t>((tokens + kCkRows - 1) / kCkRows) * W);
}
size_t rec_ws_bytes(int nseq, int64_t tokens, int W, la_dtype dt, bool backward) {
  (void)nseq;
  (void)dt;
  return sizeof(ErrRec) + (backward ? checkpoint_bytes(tokens, W) : 0);
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
  if (!workspace || !aligned256(workspace) || ws_bytes < rec_ws_bytes(p.nseq, p.tokens, p.W, dt, backward))
    return LA_ERR_INVALID_ARG;
  p.err = static_cast<ErrRec*>(workspace);
  p.tied = mode == LA_INPUT_TIED;
  cudaError_t e = cudaSuccess;
  if (!backward) {
    e = launch_rec_forward(p, dt, stream);
  } else {
    if (!p.ck) {
      RecArgs r = p;
      r.out = nullptr;
      r.s1 = nullptr;
      r.ck = p.ck = reinterpret_cast<float*>(static_cast<char*>(workspace) + sizeof(ErrRec));
      e = launch_rec_forward(r, dt, stream);
    }
    if (e == cudaSuccess) e = launch_rec_backward(p, dt, stream);
  }
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
  return la::rec_ws_bytes(num_seqs, total_tokens, W, dtype, backward != 0);
}

}  // extern "C"
