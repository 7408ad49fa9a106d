// Gated linear recurrence (ql.gl blog on Griffin/Hawk, section "Hawk"):
//     h_t = a_t h_(t-1) + b_t x_t, element by element, with
//     s = sigmoid(r), y = c softplus(lam) s, a = exp(-y), b = sqrt(1 - a^2) sigmoid(i),
// its gradients, and the one-token step.  One thread per (sequence, channel)
// walks the tokens; the backward walks the 64-token chunks last to first and
// forms each chunk's states again from the state that enters it.
#include "launch.h"

namespace ret {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// First chunk row of sequence s, which starts at flat token n.
__device__ __forceinline__ long long chunk_row(int n, int s) { return n / kGlrChunk + s; }

// Reports offsets that are not 0 <= cu[0] .. cu[nseq] = Ttot in order.
__device__ __forceinline__ void check_offsets(const SeqLayout& L, int s, unsigned* err) {
  if (L.cu == nullptr) return;
  const int a = L.cu[s], b = L.cu[s + 1];
  if ((s == 0 && a != 0) || b < a || (s == L.nseq - 1 && b != L.Ttot))
    raise_error(err, kErrDeviceData);
}

template <typename Ti, typename Th>
__global__ void __launch_bounds__(kThreads)
glr_fwd_kernel(const Ti* __restrict__ x, const Ti* __restrict__ r, const Ti* __restrict__ i,
               const float* __restrict__ lam, float c, SeqLayout L, const float* state_in,
               float* state_out, Th* h, float* chunk_states, int D, int groups, unsigned* err) {
  const int seq = blockIdx.x / groups;
  const int d = (blockIdx.x % groups) * kThreads + threadIdx.x;
  if (d == 0) check_offsets(L, seq, err);
  if (d >= D) return;
  int t0, t1;
  seq_bounds(L, seq, t0, t1);
  const float ysc = c * softplus(lam[d]);
  float st = state_in ? state_in[static_cast<size_t>(seq) * D + d] : 0.f;
  for (int t = t0; t < t1; ++t) {
    if (chunk_states && (t - t0) % kGlrChunk == 0)
      chunk_states[(chunk_row(t0, seq) + (t - t0) / kGlrChunk) * D + d] = st;
    const size_t at = static_cast<size_t>(t) * D + d;
    const float y = ysc * sigmoid(Io<Ti>::ld(r, at));
    const float b = sqrtf(-expm1f(-2.f * y)) * sigmoid(Io<Ti>::ld(i, at));
    st = fmaf(expf(-y), st, b * Io<Ti>::ld(x, at));
    Io<Th>::st(h, at, st);
  }
  if (state_out) state_out[static_cast<size_t>(seq) * D + d] = st;
}

template <typename Ti, typename Tu, typename Tg>
__global__ void __launch_bounds__(kThreads)
glr_bwd_kernel(const Ti* __restrict__ x, const Ti* __restrict__ r, const Ti* __restrict__ i,
               const float* __restrict__ lam, float c, SeqLayout L,
               const float* __restrict__ chunk_states, const Tu* __restrict__ dh,
               const float* __restrict__ d_state_out, Tg* dx, Tg* dr, Tg* di, float* d_state_in,
               float* partial, int D, int groups, unsigned* err) {
  const int seq = blockIdx.x / groups;
  const int d = (blockIdx.x % groups) * kThreads + threadIdx.x;
  if (d == 0) check_offsets(L, seq, err);
  if (d >= D) return;
  int t0, t1;
  seq_bounds(L, seq, t0, t1);
  const float ysc = c * softplus(lam[d]);
  const size_t so = static_cast<size_t>(seq) * D + d;
  float e = d_state_out ? d_state_out[so] : 0.f;
  float usum = 0.f;
  float hp[kGlrChunk];               // the state before each token of the chunk
  for (int ch = ceil_div(t1 - t0, kGlrChunk) - 1; ch >= 0; --ch) {
    const int b0 = t0 + ch * kGlrChunk, n = min(kGlrChunk, t1 - b0);
    float st = chunk_states[(chunk_row(t0, seq) + ch) * D + d];
    for (int j = 0; j < n; ++j) {
      hp[j] = st;
      const size_t at = static_cast<size_t>(b0 + j) * D + d;
      const float y = ysc * sigmoid(Io<Ti>::ld(r, at));
      const float b = sqrtf(-expm1f(-2.f * y)) * sigmoid(Io<Ti>::ld(i, at));
      st = fmaf(expf(-y), st, b * Io<Ti>::ld(x, at));
    }
    for (int j = n - 1; j >= 0; --j) {
      const size_t at = static_cast<size_t>(b0 + j) * D + d;
      const float xv = Io<Ti>::ld(x, at);
      const float sr = sigmoid(Io<Ti>::ld(r, at)), si = sigmoid(Io<Ti>::ld(i, at));
      const float y = ysc * sr, a = expf(-y), root = sqrtf(-expm1f(-2.f * y));
      const float G = Io<Tu>::ld(dh, at) + e;
      const float ratio = root > 0.f ? y / root : 0.f;
      const float gx = G * root * si;
      const float u = G * (ratio * a * a * si * xv - a * y * hp[j]);
      Io<Tg>::st(dx, at, gx);
      Io<Tg>::st(di, at, gx * xv * (1.f - si));
      Io<Tg>::st(dr, at, u * (1.f - sr));
      usum += u;
      e = a * G;
    }
  }
  if (d_state_in) d_state_in[so] = e;
  partial[so] = usum;
}

// d_lam = (sum of the partial rows) sigmoid(lam) / softplus(lam), rows in order.
__global__ void __launch_bounds__(kThreads)
glr_dlam_kernel(const float* __restrict__ partial, const float* __restrict__ lam,
                float* __restrict__ d_lam, long long rows, int D) {
  const int d = blockIdx.x * kThreads + threadIdx.x;
  if (d >= D) return;
  float s = 0.f;
  for (long long k = 0; k < rows; ++k) s += partial[k * D + d];
  // softplus(lam) -> sigmoid(lam) as both underflow
  const float sp = softplus(lam[d]);
  d_lam[d] = s * (sp > 0.f ? sigmoid(lam[d]) / sp : 1.f);
}

template <typename Ti, typename Th>
__global__ void __launch_bounds__(kThreads)
glr_step_kernel(const Ti* __restrict__ x, const Ti* __restrict__ r, const Ti* __restrict__ i,
                const float* __restrict__ lam, float c, const float* state, float* state_out,
                Th* h, int D, int groups) {
  const int d = (blockIdx.x % groups) * kThreads + threadIdx.x;
  if (d >= D) return;
  const size_t at = static_cast<size_t>(blockIdx.x / groups) * D + d;
  const float y = c * softplus(lam[d]) * sigmoid(Io<Ti>::ld(r, at));
  const float b = sqrtf(-expm1f(-2.f * y)) * sigmoid(Io<Ti>::ld(i, at));
  const float st = fmaf(expf(-y), state[at], b * Io<Ti>::ld(x, at));
  state_out[at] = st;
  if (h) Io<Th>::st(h, at, st);
}

template <typename F>
cudaError_t by_type(DType t, F&& f) {
  return t == DType::F32 ? f(float{}) : f(__nv_bfloat16{});
}

}  // namespace

long long glr_bwd_partial_rows(int nseq, long long, int) { return nseq; }

cudaError_t launch_glr_fwd(const void* x, const void* r, const void* i, DType in_t,
                           const float* lam, float c, const SeqLayout& L, const float* state_in,
                           float* state_out, void* h, DType h_t, float* chunk_states, int D,
                           unsigned* err, cudaStream_t s) {
  const int groups = (D + kThreads - 1) / kThreads;
  const long long blocks = static_cast<long long>(groups) * L.nseq;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return by_type(in_t, [&](auto ti) {
    return by_type(h_t, [&](auto th) {
      using Ti = decltype(ti);
      using Th = decltype(th);
      glr_fwd_kernel<Ti, Th><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
          static_cast<const Ti*>(x), static_cast<const Ti*>(r), static_cast<const Ti*>(i), lam, c,
          L, state_in, state_out, static_cast<Th*>(h), chunk_states, D, groups, err);
      return cudaGetLastError();
    });
  });
}

cudaError_t launch_glr_bwd(const void* x, const void* r, const void* i, DType in_t,
                           const float* lam, float c, const SeqLayout& L,
                           const float* chunk_states, const void* d_h, DType dh_t,
                           const float* d_state_out, void* dx, void* dr, void* di, DType g_t,
                           float* d_lam, float* d_state_in, float* partial, int D, unsigned* err,
                           cudaStream_t s) {
  const int groups = (D + kThreads - 1) / kThreads;
  const long long blocks = static_cast<long long>(groups) * L.nseq;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const cudaError_t e = by_type(in_t, [&](auto ti) {
    return by_type(dh_t, [&](auto tu) {
      return by_type(g_t, [&](auto tg) {
        using Ti = decltype(ti);
        using Tu = decltype(tu);
        using Tg = decltype(tg);
        glr_bwd_kernel<Ti, Tu, Tg><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
            static_cast<const Ti*>(x), static_cast<const Ti*>(r), static_cast<const Ti*>(i), lam,
            c, L, chunk_states, static_cast<const Tu*>(d_h), d_state_out, static_cast<Tg*>(dx),
            static_cast<Tg*>(dr), static_cast<Tg*>(di), d_state_in, partial, D, groups, err);
        return cudaGetLastError();
      });
    });
  });
  if (e != cudaSuccess) return e;
  glr_dlam_kernel<<<groups, kThreads, 0, s>>>(partial, lam, d_lam,
                                              glr_bwd_partial_rows(L.nseq, L.Ttot, D), D);
  return cudaGetLastError();
}

cudaError_t launch_glr_step(const void* x, const void* r, const void* i, DType in_t,
                            const float* lam, float c, const float* state, float* state_out,
                            void* h, DType h_t, int N, int D, cudaStream_t s) {
  const int groups = (D + kThreads - 1) / kThreads;
  const long long blocks = static_cast<long long>(groups) * N;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return by_type(in_t, [&](auto ti) {
    return by_type(h_t, [&](auto th) {
      using Ti = decltype(ti);
      using Th = decltype(th);
      glr_step_kernel<Ti, Th><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
          static_cast<const Ti*>(x), static_cast<const Ti*>(r), static_cast<const Ti*>(i), lam, c,
          state, state_out, static_cast<Th*>(h), D, groups);
      return cudaGetLastError();
    });
  });
}

}  // namespace ret
