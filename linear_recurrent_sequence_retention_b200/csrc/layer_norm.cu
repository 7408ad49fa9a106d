// Layer norm over the last dimension and its gradients (formulas in
// include/retention.h).  HBM-bound: the forward reads x and writes y once, the
// gradients read x and d_y and write dx once.
//
// Forward: a row belongs to one warp (up to 1024 channels) or one block and stays in
// registers between its two statistics passes and the output.
//
// Gradients: blocks stay and walk rows, so that each thread keeps its channels'
// weight and the sums for d_weight and d_bias in registers; the rows to come are on their
// way to shared memory meanwhile.  The blocks' sums go to the workspace and a second
// kernel adds them in a fixed order.
#include "norm_common.cuh"

namespace ret {
namespace {

using namespace norm;

// ---- forward -------------------------------------------------------------------

template <typename Tx, typename Ty, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
ln_fwd_kernel(const Tx* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
              float eps, float invD, Ty* __restrict__ y, float* __restrict__ mean,
              float* __restrict__ rstd, int ntok, int D) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;        // rows of a block
  __shared__ float part[2 * (TPR / 32)];
  const int t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / TPR;
  if (TPR <= 32 && row >= ntok) return;                   // whole warps
  const size_t base = static_cast<size_t>(row) * D;
  Raw8<Tx> raw[NV];
  float s[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * 8;
    if (c < D) raw[k] = load8(x + base + c);
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if ((k * TPR + t) * 8 < D) {
      float v[8];
      unpack(raw[k], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[e];
    }
  row_sum<TPR>(s, part, 0);
  const float mu = s[0] * invD;
  s[0] = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if ((k * TPR + t) * 8 < D) {
      float v[8];
      unpack(raw[k], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] = fmaf(v[e] - mu, v[e] - mu, s[0]);
    }
  row_sum<TPR>(s, part, 1);
  const float rs = inv_std(s[0] * invD, eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * 8;
    if (c < D) {
      float v[8], wv[8], bv[8];
      unpack(raw[k], v);
      weights8(w, c, 1.f, wv);
      weights8(b, c, 0.f, bv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - mu) * rs, wv[e], bv[e]);
      store8(y + base + c, v);
    }
  }
  if (t == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
}

// Any width, any types: one channel at a time.
template <int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
ln_fwd_any_kernel(Any x, const float* __restrict__ w, const float* __restrict__ b, float eps,
                  float invD, AnyOut y, float* __restrict__ mean, float* __restrict__ rstd, int ntok, int D) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  __shared__ float part[2 * (TPR / 32)];
  const int t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / TPR;
  if (TPR <= 32 && row >= ntok) return;
  const size_t base = static_cast<size_t>(row) * D;
  float v[NV];
  float s[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = k * TPR + t;
    v[k] = c < D ? x.ld(base + c) : 0.f;
    s[0] += v[k];
  }
  row_sum<TPR>(s, part, 0);
  const float mu = s[0] * invD;
  s[0] = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (k * TPR + t < D) s[0] = fmaf(v[k] - mu, v[k] - mu, s[0]);
  row_sum<TPR>(s, part, 1);
  const float rs = inv_std(s[0] * invD, eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = k * TPR + t;
    if (c < D) y.st(base + c, fmaf((v[k] - mu) * rs, w ? w[c] : 1.f, b ? b[c] : 0.f));
  }
  if (t == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
}

// ---- gradients -------------------------------------------------------------------

// A block holds several rows where they are short; blocks of 64 registers per thread fill half
// an SM's threads.
#ifndef BNV
#define BNV 2
#endif
constexpr int bwd_threads(int TPR) { return TPR < 256 ? 256 : TPR; }
constexpr int bwd_blocks_per_sm(int TPR, int NV) { return TPR > 256 ? 1 : NV > 2 ? 1 : NV == 2 ? 2 : 4; }

// 16-byte units of a thread and stage, and the stages (rows on their way, and one in use).
template <typename Tx, typename Tu> constexpr int bwd_units(int NV) {
  return NV * (Raw8<Tx>::kU + Raw8<Tu>::kU);
}
template <typename Tx, typename Tu> constexpr int bwd_stages(int TPR, int NV) {
  return stages(bwd_units<Tx, Tu>(NV) * bwd_threads(TPR) * 16, bwd_blocks_per_sm(TPR, NV));
}

// Adds the sums of the block's row groups (`acc`, groups x D) in order.
template <int TPR>
__device__ __forceinline__ void write_partial(const float* acc, float* out, int D) {
  constexpr int kGroups = bwd_threads(TPR) / TPR;
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += bwd_threads(TPR)) {
    float v = acc[c];
#pragma unroll
    for (int g = 1; g < kGroups; ++g) v += acc[g * D + c];
    out[c] = v;
  }
  __syncthreads();
}

template <typename Tx, typename Tu, typename Tg, int TPR, int NV>
__global__ void __launch_bounds__(bwd_threads(TPR), bwd_blocks_per_sm(TPR, NV))
ln_bwd_kernel(const Tx* __restrict__ x, const Tu* __restrict__ dy, const float* __restrict__ mean,
              const float* __restrict__ rstd, const float* __restrict__ w, Tg* __restrict__ dx,
              float* __restrict__ partial, int ntok, int D) {
  constexpr int kThreads = bwd_threads(TPR), kGroups = kThreads / TPR;
  constexpr int kUx = Raw8<Tx>::kU, kUu = Raw8<Tu>::kU;
  constexpr int kUnits = bwd_units<Tx, Tu>(NV), kStages = bwd_stages<Tx, Tu>(TPR, NV);
  extern __shared__ __align__(16) char smem[];
  __shared__ float parts[kGroups][2 * 2 * (TPR > 32 ? TPR / 32 : 1)];
  const int group = threadIdx.x / TPR;
  float* part = parts[group];
  uint4* ring = reinterpret_cast<uint4*>(smem) + threadIdx.x;
  const int t = threadIdx.x % TPR;
  const int step = gridDim.x * kGroups;
  int row = blockIdx.x * kGroups + group;
  const auto fetch = [&](int r, int stage) {
    if (r < ntok) {
      uint4* s = ring + stage * (kUnits * kThreads);
      const size_t base = static_cast<size_t>(r) * D;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (k * TPR + t) * 8;
        if (c < D) {
          copy8(s + k * kUx * kThreads, kThreads, x + base + c);
          copy8(s + (NV * kUx + k * kUu) * kThreads, kThreads, dy + base + c);
        }
      }
    }
    copies_commit();
  };
  // 64-bit: the last rows of a stride may pass 2^31
  const auto ahead = [&](int n) {
    const long long r = row + static_cast<long long>(n) * step;
    return r < ntok ? static_cast<int>(r) : ntok;
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(ahead(k), k);
  float wv[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * 8;
    if (c < D) weights8(w, c, 1.f, wv[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c >= D) wv[k][e] = 0.f;
      dw[k][e] = db[k][e] = 0.f;
    }
  }
  float mu = row < ntok ? mean[row] : 0.f, rs = row < ntok ? rstd[row] : 0.f;
  const float invD = 1.0f / D;
  int use = 0, fill = kStages - 1;
  for (int it = 0; row < ntok; ++it) {
    fetch(ahead(kStages - 1), fill);
    const int next = ahead(1);
    const float mu_next = next < ntok ? mean[next] : 0.f, rs_next = next < ntok ? rstd[next] : 0.f;
    copies_wait<kStages - 1>();
    const uint4* s = ring + use * (kUnits * kThreads);
    Raw8<Tx> xr[NV];
    Raw8<Tu> ur[NV];
    float sum[2] = {0.f, 0.f};            // of n, and of n (x - mean)
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * TPR + t) * 8 < D) {
        xr[k] = read8<Tx>(s + k * kUx * kThreads, kThreads);
        ur[k] = read8<Tu>(s + (NV * kUx + k * kUu) * kThreads, kThreads);
        float xv[8], uv[8];
        unpack(xr[k], xv);
        unpack(ur[k], uv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = uv[e] * wv[k][e];
          sum[0] += n;
          sum[1] = fmaf(n, xv[e] - mu, sum[1]);
        }
      }
    row_sum<TPR>(sum, part, it, group);
    const float m1 = -rs * sum[0] * invD, m2 = -rs * rs * sum[1] * invD;
    const size_t base = static_cast<size_t>(row) * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * 8;
      if (c < D) {
        float xv[8], uv[8], g[8];
        unpack(xr[k], xv);
        unpack(ur[k], uv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = (xv[e] - mu) * rs;
          dw[k][e] = fmaf(uv[e], xh, dw[k][e]);
          db[k][e] += uv[e];
          g[e] = fmaf(xh, m2, fmaf(uv[e] * wv[k][e], rs, m1));
        }
        store8(dx + base + c, g);
      }
    }
    fill = use;
    use = use + 1 == kStages ? 0 : use + 1;
    row = next;
    mu = mu_next;
    rs = rs_next;
  }
  if (!partial) return;
  copies_wait<0>();
  float* mine = partial + static_cast<size_t>(blockIdx.x) * D;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * 8;
      if (c < D) {
        store8(mine + c, dw[k]);
        store8(mine + static_cast<size_t>(gridDim.x) * D + c, db[k]);
      }
    }
  } else {
    float* acc = reinterpret_cast<float*>(smem);
    float* own = acc + group * D;
    __syncthreads();                      // every group has read its rows from the ring
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * TPR + t) * 8 < D) store8(own + (k * TPR + t) * 8, dw[k]);
    write_partial<TPR>(acc, mine, D);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * TPR + t) * 8 < D) store8(own + (k * TPR + t) * 8, db[k]);
    write_partial<TPR>(acc, mine + static_cast<size_t>(gridDim.x) * D, D);
  }
}

// Any width, any types: one channel at a time.
template <int TPR, int NV>
__global__ void __launch_bounds__(bwd_threads(TPR))
ln_bwd_any_kernel(Any x, Any dy, const float* __restrict__ mean, const float* __restrict__ rstd,
                  const float* __restrict__ w, AnyOut dx, float* __restrict__ partial, int ntok,
                  int D) {
  constexpr int kThreads = bwd_threads(TPR), kGroups = kThreads / TPR;
  extern __shared__ __align__(16) char smem[];
  __shared__ float parts[kGroups][2 * 2 * (TPR > 32 ? TPR / 32 : 1)];
  const int group = threadIdx.x / TPR;
  float* part = parts[group];
  const int t = threadIdx.x % TPR;
  const long long step = static_cast<long long>(gridDim.x) * kGroups;
  float dw[NV], db[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) dw[k] = db[k] = 0.f;
  const float invD = 1.0f / D;
  int it = 0;
  for (long long row = blockIdx.x * kGroups + group; row < ntok; row += step, ++it) {
    const size_t base = static_cast<size_t>(row) * D;
    const float mu = mean[row], rs = rstd[row];
    float xv[NV], uv[NV], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = k * TPR + t;
      xv[k] = c < D ? x.ld(base + c) : mu;
      uv[k] = c < D ? dy.ld(base + c) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = k * TPR + t;
      const float n = uv[k] * (w && c < D ? w[c] : 1.f);
      sum[0] += n;
      sum[1] = fmaf(n, xv[k] - mu, sum[1]);
    }
    row_sum<TPR>(sum, part, it, group);
    const float m1 = sum[0] * invD, m2 = sum[1] * invD * rs;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = k * TPR + t;
      const float xh = (xv[k] - mu) * rs;
      dw[k] = fmaf(uv[k], xh, dw[k]);
      db[k] += uv[k];
      if (c < D) dx.st(base + c, rs * (fmaf(uv[k], w ? w[c] : 1.f, -m1) - xh * m2));
    }
  }
  if (!partial) return;
  float* mine = partial + static_cast<size_t>(blockIdx.x) * D;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = k * TPR + t;
      if (c < D) {
        mine[c] = dw[k];
        mine[static_cast<size_t>(gridDim.x) * D + c] = db[k];
      }
    }
  } else {
    float* acc = reinterpret_cast<float*>(smem);
    float* own = acc + group * D;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (k * TPR + t < D) own[k * TPR + t] = dw[k];
    write_partial<TPR>(acc, mine, D);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (k * TPR + t < D) own[k * TPR + t] = db[k];
    write_partial<TPR>(acc, mine + static_cast<size_t>(gridDim.x) * D, D);
  }
}

// ---- which variant -----------------------------------------------------------------

// Threads and values per thread of a row; D <= tpr * nv * vec.
struct Shape {
  int vec, tpr, nv;
};

// Forward: a warp per row up to 1024 channels, otherwise a block with up to four vectors per
// thread; few rows (at most two per SM) get a thread for every vector or two instead, since the
// row's own latency counts then.
Shape fwd_shape(int ntok, int D) {
  if (D % 8 == 0) {
    const int n = D / 8;
    const bool few = ntok <= 2 * kSms;
    if (n <= 32) return {8, 32, 1};
    if (n <= 64) return {8, 32, 2};
    if (n <= 128 && !few) return {8, 32, 4};
    if (n <= 256) return {8, 128, 2};
#ifdef LNF
    if (n <= 512) return few ? Shape{8, 512, 1} : Shape{8, LNF, 512/LNF};
#endif
    if (n <= 512) return few ? Shape{8, 512, 1} : Shape{8, 128, 4};
    if (n <= 1024) return few ? Shape{8, 512, 2} : Shape{8, 256, 4};
    return {8, 512, 4};
  }
  if (D <= 256) return {1, 32, 8};
  if (D <= 1024) return {1, 128, 8};
  if (D <= 4096) return {1, 256, 16};
  return {1, 512, 32};
}
// Gradients: one vector per thread where a block can be that large (three values stay in
// registers for each channel).
Shape bwd_shape(int D) {
  if (D % 8 == 0) {
    const int n = D / 8;
    int tpr = 32, nv = BNV;
    while (tpr * nv < n && tpr < 512) tpr *= 2;
    if (tpr * nv < n) nv = n <= 1024 ? 2 : 4;
    return {8, tpr, nv};
  }
  if (D <= 256) return {1, 32, 8};
  if (D <= 1024) return {1, 128, 8};
  if (D <= 4096) return {1, 256, 16};
  return {1, 512, 32};
}

template <int T, int N> struct Pick {
  static constexpr int tpr = T, nv = N;
};
template <typename F>
cudaError_t with_shape(const Shape& s, F&& f) {
  switch (s.tpr * 64 + s.nv) {
    case 32 * 64 + 1: return f(Pick<32, 1>{});
    case 32 * 64 + 2: return f(Pick<32, 2>{});
    case 32 * 64 + 4: return f(Pick<32, 4>{});
    case 32 * 64 + 8: return f(Pick<32, 8>{});
    case 64 * 64 + 1: return f(Pick<64, 1>{});
    case 64 * 64 + 2: return f(Pick<64, 2>{});
    case 64 * 64 + 4: return f(Pick<64, 4>{});
    case 128 * 64 + 1: return f(Pick<128, 1>{});
    case 128 * 64 + 2: return f(Pick<128, 2>{});
    case 128 * 64 + 4: return f(Pick<128, 4>{});
    case 128 * 64 + 8: return f(Pick<128, 8>{});
    case 256 * 64 + 1: return f(Pick<256, 1>{});
    case 256 * 64 + 2: return f(Pick<256, 2>{});
    case 256 * 64 + 4: return f(Pick<256, 4>{});
    case 256 * 64 + 16: return f(Pick<256, 16>{});
    case 512 * 64 + 1: return f(Pick<512, 1>{});
    case 512 * 64 + 2: return f(Pick<512, 2>{});
    case 512 * 64 + 4: return f(Pick<512, 4>{});
    case 512 * 64 + 32: return f(Pick<512, 32>{});
    case 1024 * 64 + 1: return f(Pick<1024, 1>{});
  }
  return cudaErrorInvalidConfiguration;
}
// Compiles only what a shape table can name.
constexpr bool fwd_vec(int tpr, int nv) {
  return (tpr == 32 && nv <= 4) || (tpr == 128 && nv >= 2 && nv <= 4) || (tpr == 256 && (nv == 2 || nv == 4)) ||
         (tpr == 512 && nv <= 4);
}
constexpr bool bwd_vec(int tpr, int nv) { return tpr <= 512 && (nv == BNV || (tpr == 512 && nv >= 2 && nv <= 4)); }
constexpr bool any_width(int tpr, int nv) {
  return (tpr <= 128 && nv == 8) || (tpr == 256 && nv == 16) || (tpr == 512 && nv == 32);
}

int bwd_blocks(const Shape& s, int ntok) {
  const int groups = bwd_threads(s.tpr) / s.tpr;
  const int per_sm = s.vec == 1 ? (s.tpr > 256 ? 1 : 4) : bwd_blocks_per_sm(s.tpr, s.nv);
  const int need = (ntok + groups - 1) / groups;
  return need < kSms * per_sm ? need : kSms * per_sm;
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const void* x, DType x_t, const float* w, const float* b,
                                  float eps, void* y, DType y_t, float* mean, float* rstd,
                                  int ntok, int D, cudaStream_t s) {
  const Shape sh = fwd_shape(ntok, D);
  const float invD = 1.0f / static_cast<float>(D);
  const int rows = sh.tpr < 128 ? 128 / sh.tpr : 1;
  const unsigned blocks = static_cast<unsigned>((ntok + static_cast<long long>(rows) - 1) / rows);
  const int threads = sh.tpr < 128 ? 128 : sh.tpr;
  return with_shape(sh, [&](auto p) {
    constexpr int T = decltype(p)::tpr, N = decltype(p)::nv;
    if (sh.vec == 1) {
      if constexpr (any_width(T, N)) {
        ln_fwd_any_kernel<T, N><<<blocks, threads, 0, s>>>(Any{x, x_t == DType::F32}, w, b, eps,
                                                          invD, AnyOut{y, y_t == DType::F32}, mean, rstd,
                                                          ntok, D);
        return cudaGetLastError();
      }
    } else if constexpr (fwd_vec(T, N)) {
      return by_type(x_t, [&](auto tx) {
        return by_type(y_t, [&](auto ty) {
          using Tx = decltype(tx);
          using Ty = decltype(ty);
          ln_fwd_kernel<Tx, Ty, T, N><<<blocks, threads, 0, s>>>(
              static_cast<const Tx*>(x), w, b, eps, invD, static_cast<Ty*>(y), mean, rstd, ntok, D);
          return cudaGetLastError();
        });
      });
    }
    return cudaErrorInvalidConfiguration;
  });
}

int layer_norm_bwd_partial_rows(int ntok, int D) { return bwd_blocks(bwd_shape(D), ntok); }

cudaError_t launch_layer_norm_bwd(const void* x, DType x_t, const void* dy, DType dy_t,
                                  const float* mean, const float* rstd, const float* w, void* dx,
                                  DType dx_t, float* dw, float* db, float* partial, int ntok,
                                  int D, cudaStream_t s) {
  const Shape sh = bwd_shape(D);
  const int blocks = bwd_blocks(sh, ntok);
  float* part = dw ? partial : nullptr;
  cudaError_t e = cudaSuccess;
  if (blocks > 0)
    e = with_shape(sh, [&](auto p) {
      constexpr int T = decltype(p)::tpr, N = decltype(p)::nv;
      constexpr int kThreads = bwd_threads(T);
      const size_t sums = kThreads / T > 1 ? static_cast<size_t>(kThreads / T) * D * sizeof(float) : 0;
      if (sh.vec == 1) {
        if constexpr (any_width(T, N)) {
          const cudaError_t a = allow_smem(ln_bwd_any_kernel<T, N>, sums);
          if (a != cudaSuccess) return a;
          ln_bwd_any_kernel<T, N><<<blocks, kThreads, sums, s>>>(
              Any{x, x_t == DType::F32}, Any{dy, dy_t == DType::F32}, mean, rstd, w,
              AnyOut{dx, dx_t == DType::F32}, part, ntok, D);
          return cudaGetLastError();
        }
      } else if constexpr (bwd_vec(T, N)) {
        return by_type(x_t, [&](auto tx) {
          return by_type(dy_t, [&](auto tu) {
            return by_type(dx_t, [&](auto tg) {
              using Tx = decltype(tx);
              using Tu = decltype(tu);
              using Tg = decltype(tg);
              const size_t ring = static_cast<size_t>(bwd_stages<Tx, Tu>(T, N)) *
                                  bwd_units<Tx, Tu>(N) * kThreads * sizeof(uint4);
              const size_t smem = ring > sums ? ring : sums;
              const cudaError_t a = allow_smem(ln_bwd_kernel<Tx, Tu, Tg, T, N>, smem);
              if (a != cudaSuccess) return a;
              ln_bwd_kernel<Tx, Tu, Tg, T, N><<<blocks, kThreads, smem, s>>>(
                  static_cast<const Tx*>(x), static_cast<const Tu*>(dy), mean, rstd, w,
                  static_cast<Tg*>(dx), part, ntok, D);
              return cudaGetLastError();
            });
          });
        });
      }
      return cudaErrorInvalidConfiguration;
    });
  if (e != cudaSuccess || !dw) return e;
  return sum_rows(partial, dw, db, blocks, D, s);
}

}  // namespace ret
