// Layer norm, its gradients, and the gradients of the per-head GroupNorm +
// Swish gate (formulas in include/retention.h).  One warp per row (a token, or
// a token's head); the weights' gradients are summed by one thread per column.
#include "launch.h"

namespace ret {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float v) {
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

template <typename T>
__device__ __forceinline__ void row_stats(const T* x, size_t base, int D, int lane, float eps,
                                          float& mean, float& rstd) {
  float s = 0.f;
  for (int c = lane; c < D; c += 32) s += Io<T>::ld(x, base + c);
  mean = warp_sum(s) / D;
  float q = 0.f;
  for (int c = lane; c < D; c += 32) {
    const float v = Io<T>::ld(x, base + c) - mean;
    q += v * v;
  }
  rstd = 1.0f / sqrtf(warp_sum(q) / D + eps);
}

template <typename Tx, typename Ty>
__global__ void __launch_bounds__(kWarps * 32)
layer_norm_fwd_kernel(const Tx* __restrict__ x, const float* __restrict__ w,
                      const float* __restrict__ b, float eps, Ty* __restrict__ y, float* mean,
                      float* rstd, int ntok, int D) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= ntok) return;
  const size_t base = static_cast<size_t>(row) * D;
  float mu, rs;
  row_stats(x, base, D, lane, eps, mu, rs);
  for (int c = lane; c < D; c += 32) {
    float v = (Io<Tx>::ld(x, base + c) - mu) * rs;
    if (w) v *= w[c];
    if (b) v += b[c];
    Io<Ty>::st(y, base + c, v);
  }
  if (lane == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
}

template <typename Tx, typename Tu, typename Tg>
__global__ void __launch_bounds__(kWarps * 32)
layer_norm_dx_kernel(const Tx* __restrict__ x, const Tu* __restrict__ dy,
                     const float* __restrict__ mean, const float* __restrict__ rstd,
                     const float* __restrict__ w, Tg* __restrict__ dx, int ntok, int D) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= ntok) return;
  const size_t base = static_cast<size_t>(row) * D;
  const float mu = mean[row], rs = rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int c = lane; c < D; c += 32) {
    const float n = Io<Tu>::ld(dy, base + c) * (w ? w[c] : 1.f);
    s1 += n;
    s2 += n * (Io<Tx>::ld(x, base + c) - mu) * rs;
  }
  s1 = warp_sum(s1) / D;
  s2 = warp_sum(s2) / D;
  for (int c = lane; c < D; c += 32) {
    const float n = Io<Tu>::ld(dy, base + c) * (w ? w[c] : 1.f);
    const float xh = (Io<Tx>::ld(x, base + c) - mu) * rs;
    Io<Tg>::st(dx, base + c, rs * (n - s1 - xh * s2));
  }
}

template <typename Tx, typename Tu>
__global__ void layer_norm_dw_kernel(const Tx* __restrict__ x, const Tu* __restrict__ dy,
                                     const float* __restrict__ mean,
                                     const float* __restrict__ rstd, float* dw, float* db,
                                     int ntok, int D) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= D) return;
  float sw = 0.f, sb = 0.f;
  for (int n = 0; n < ntok; ++n) {
    const size_t at = static_cast<size_t>(n) * D + c;
    const float g = Io<Tu>::ld(dy, at);
    sw += g * (Io<Tx>::ld(x, at) - mean[n]) * rstd[n];
    sb += g;
  }
  dw[c] = sw;
  db[c] = sb;
}

template <typename To, typename Ti, typename Tg>
__global__ void __launch_bounds__(kWarps * 32)
norm_gate_dx_kernel(const To* __restrict__ o, const Ti* __restrict__ g,
                    const Ti* __restrict__ dy, const float* __restrict__ w,
                    const float* __restrict__ b, float eps, Tg* __restrict__ d_o,
                    Tg* __restrict__ d_g, long long nrows, int H, int dv) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= nrows) return;
  const int h0 = static_cast<int>(row % H) * dv;
  const size_t base = static_cast<size_t>(row) * dv;
  float mu, rs;
  row_stats(o, base, dv, lane, eps, mu, rs);
  float s1 = 0.f, s2 = 0.f;
  for (int c = lane; c < dv; c += 32) {
    const float gv = Io<Ti>::ld(g, base + c);
    const float n = Io<Ti>::ld(dy, base + c) * gv * sigmoid(gv) * (w ? w[h0 + c] : 1.f);
    s1 += n;
    s2 += n * (Io<To>::ld(o, base + c) - mu) * rs;
  }
  s1 = warp_sum(s1) / dv;
  s2 = warp_sum(s2) / dv;
  for (int c = lane; c < dv; c += 32) {
    const float gv = Io<Ti>::ld(g, base + c), u = Io<Ti>::ld(dy, base + c);
    const float sg = sigmoid(gv), wc = w ? w[h0 + c] : 1.f;
    const float xh = (Io<To>::ld(o, base + c) - mu) * rs;
    const float t = fmaf(xh, wc, b ? b[h0 + c] : 0.f);
    Io<Tg>::st(d_g, base + c, u * t * sg * (1.f + gv * (1.f - sg)));
    Io<Tg>::st(d_o, base + c, rs * (u * gv * sg * wc - s1 - xh * s2));
  }
}

// One block per head; thread c < dv sums its column, the block shares the row statistics.
template <typename To, typename Ti>
__global__ void norm_gate_dw_kernel(const To* __restrict__ o, const Ti* __restrict__ g,
                                    const Ti* __restrict__ dy, float eps, float* dw, float* db,
                                    int ntok, int H, int dv) {
  __shared__ float st[2];
  const int h = blockIdx.x, c = threadIdx.x;
  float sw = 0.f, sb = 0.f;
  for (int n = 0; n < ntok; ++n) {
    const size_t base = (static_cast<size_t>(n) * H + h) * dv;
    __syncthreads();
    if (c < 32) {
      float mu, rs;
      row_stats(o, base, dv, c, eps, mu, rs);
      st[0] = mu;
      st[1] = rs;
    }
    __syncthreads();
    if (c < dv) {
      const float gv = Io<Ti>::ld(g, base + c);
      const float dt = Io<Ti>::ld(dy, base + c) * gv * sigmoid(gv);
      sw += dt * (Io<To>::ld(o, base + c) - st[0]) * st[1];
      sb += dt;
    }
  }
  if (c < dv) {
    dw[h * dv + c] = sw;
    db[h * dv + c] = sb;
  }
}

template <typename F>
cudaError_t by_type(DType t, F&& f) {
  return t == DType::F32 ? f(float{}) : f(__nv_bfloat16{});
}

unsigned warp_blocks(long long rows) { return static_cast<unsigned>((rows + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_layer_norm_fwd(const void* x, DType x_t, const float* w, const float* b,
                                  float eps, void* y, DType y_t, float* mean, float* rstd,
                                  int ntok, int D, cudaStream_t s) {
  return by_type(x_t, [&](auto tx) {
    return by_type(y_t, [&](auto ty) {
      using Tx = decltype(tx);
      using Ty = decltype(ty);
      layer_norm_fwd_kernel<Tx, Ty><<<warp_blocks(ntok), kWarps * 32, 0, s>>>(
          static_cast<const Tx*>(x), w, b, eps, static_cast<Ty*>(y), mean, rstd, ntok, D);
      return cudaGetLastError();
    });
  });
}

int layer_norm_bwd_partial_rows(int, int) { return 0; }

cudaError_t launch_layer_norm_bwd(const void* x, DType x_t, const void* dy, DType dy_t,
                                  const float* mean, const float* rstd, const float* w, void* dx,
                                  DType dx_t, float* dw, float* db, float*, int ntok, int D,
                                  cudaStream_t s) {
  return by_type(x_t, [&](auto tx) {
    return by_type(dy_t, [&](auto tu) {
      using Tx = decltype(tx);
      using Tu = decltype(tu);
      cudaError_t e = cudaSuccess;
      if (ntok > 0)
        e = by_type(dx_t, [&](auto tg) {
          using Tg = decltype(tg);
          layer_norm_dx_kernel<Tx, Tu, Tg><<<warp_blocks(ntok), kWarps * 32, 0, s>>>(
              static_cast<const Tx*>(x), static_cast<const Tu*>(dy), mean, rstd, w,
              static_cast<Tg*>(dx), ntok, D);
          return cudaGetLastError();
        });
      if (e != cudaSuccess || !dw) return e;
      layer_norm_dw_kernel<Tx, Tu><<<(D + 127) / 128, 128, 0, s>>>(
          static_cast<const Tx*>(x), static_cast<const Tu*>(dy), mean, rstd, dw, db, ntok, D);
      return cudaGetLastError();
    });
  });
}

int norm_gate_bwd_partial_rows(int, int, int) { return 0; }

cudaError_t launch_norm_gate_bwd(const void* o, DType o_t, const void* g, const void* dy,
                                 DType g_t, const float* w, const float* b, float eps, void* d_o,
                                 void* d_g, DType grad_t, float* dw, float* db, float*, int ntok,
                                 int H, int dv, cudaStream_t s) {
  const long long rows = static_cast<long long>(ntok) * H;
  if ((rows + kWarps - 1) / kWarps > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return by_type(o_t, [&](auto to) {
    return by_type(g_t, [&](auto ti) {
      using To = decltype(to);
      using Ti = decltype(ti);
      cudaError_t e = cudaSuccess;
      if (ntok > 0)
        e = by_type(grad_t, [&](auto tg) {
          using Tg = decltype(tg);
          norm_gate_dx_kernel<To, Ti, Tg><<<warp_blocks(rows), kWarps * 32, 0, s>>>(
              static_cast<const To*>(o), static_cast<const Ti*>(g), static_cast<const Ti*>(dy), w,
              b, eps, static_cast<Tg*>(d_o), static_cast<Tg*>(d_g), rows, H, dv);
          return cudaGetLastError();
        });
      if (e != cudaSuccess || !dw) return e;
      norm_gate_dw_kernel<To, Ti><<<H, (dv + 31) / 32 * 32, 0, s>>>(
          static_cast<const To*>(o), static_cast<const Ti*>(g), static_cast<const Ti*>(dy), eps,
          dw, db, ntok, H, dv);
      return cudaGetLastError();
    });
  });
}

}  // namespace ret
