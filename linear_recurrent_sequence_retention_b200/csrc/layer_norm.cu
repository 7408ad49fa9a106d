// Layer norm over the last dimension and its gradients (formulas in
// include/retention.h).  HBM-bound: the forward reads x and writes y once, the
// gradients read x and d_y and write dx once.  Measured at 16384 x 4096 bf16: forward
// 0.047 ms (5.7 TB/s, 87 % of the measured copy rate), gradients 0.077 ms (5.2 TB/s, 80 %), of
// which 4.5 us are the sum of the weights' partial gradients.
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

// Vectors of four channels: with eight (bf16) the float32 weights of a thread are 32 bytes apart
// from its neighbour's, twice the cache lines per access.
constexpr int kFwdVec = 4;

template <typename Tx, typename Ty, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
ln_fwd_kernel(const Tx* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
              float eps, float invD, Ty* __restrict__ y, float* __restrict__ mean,
              float* __restrict__ rstd, int ntok, int D) {
  constexpr int VEC = kFwdVec;
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;        // rows of a block
  __shared__ float part[2 * (TPR / 32)];
  const int t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / TPR;
  if (TPR <= 32 && row >= ntok) return;                   // whole warps
  const size_t base = static_cast<size_t>(row) * D;
  Raw<Tx, VEC> raw[NV];
  float s[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (c < D) raw[k] = load<VEC>(x + base + c);
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if ((k * TPR + t) * VEC < D) {
      float v[VEC];
      unpack(raw[k], v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += v[e];
    }
  row_sum<TPR>(s, part, 0);
  const float mu = s[0] * invD;
  s[0] = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if ((k * TPR + t) * VEC < D) {
      float v[VEC];
      unpack(raw[k], v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] = fmaf(v[e] - mu, v[e] - mu, s[0]);
    }
  row_sum<TPR>(s, part, 1);
  const float rs = inv_std(s[0] * invD, eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (c < D) {
      float v[VEC], wv[VEC], bv[VEC];
      unpack(raw[k], v);
      weights(w, c, 1.f, wv);
      weights(b, c, 0.f, bv);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf((v[e] - mu) * rs, wv[e], bv[e]);
      store(y + base + c, v);
    }
  }
  if (t == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = rs;
  }
}

// Any width: one channel at a time.  Bound by the latency of its loads, of which nothing is on its way
// ahead: 8 us at 4099 x 1001 bf16, 16 MB.
template <typename Tx, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
ln_fwd_any_kernel(const Tx* __restrict__ x, const float* __restrict__ w,
                  const float* __restrict__ b, float eps, float invD, AnyOut y,
                  float* __restrict__ mean, float* __restrict__ rstd, int ntok, int D) {
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
    v[k] = c < D ? Io<Tx>::ld(x, base + c) : 0.f;
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

// A block holds several rows where they are short.
constexpr int bwd_threads(int TPR) { return TPR < 256 ? 256 : TPR; }
constexpr int bwd_blocks_per_sm(int TPR) { return TPR > 256 ? 1 : 2; }      // 128 registers
// Bytes of a stage (a row of x and of d_y per row group, and its statistics), and the stages (rows
// on their way, and one in use).  CH: channels of a thread.
template <typename Tx, typename Tu> constexpr int bwd_stage_bytes(int TPR, int CH) {
  return bwd_threads(TPR) * CH * static_cast<int>(sizeof(Tx) + sizeof(Tu)) + bwd_threads(TPR) / 32 * 8;
}
template <typename Tx, typename Tu> constexpr int bwd_stages(int TPR, int CH) {
  return stages(bwd_stage_bytes<Tx, Tu>(TPR, CH), bwd_blocks_per_sm(TPR));
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

template <typename Tx, typename Tu, typename Tg, int TPR, int CH>
__global__ void __launch_bounds__(bwd_threads(TPR), bwd_blocks_per_sm(TPR))
ln_bwd_kernel(const Tx* __restrict__ x, const Tu* __restrict__ dy, const float* __restrict__ mean,
              const float* __restrict__ rstd, const float* __restrict__ w, Tg* __restrict__ dx,
              float* __restrict__ partial, int ntok, int D) {
  constexpr int VEC = vec_of<Tx, Tu, Tg>(), NV = CH / VEC;
  constexpr int kThreads = bwd_threads(TPR), kGroups = kThreads / TPR;
  constexpr int kStages = bwd_stages<Tx, Tu>(TPR, CH), kStage = bwd_stage_bytes<Tx, Tu>(TPR, CH);
  constexpr int kDy = kThreads * CH * static_cast<int>(sizeof(Tx));           // offsets in a stage
  constexpr int kStats = kDy + kThreads * CH * static_cast<int>(sizeof(Tu));
  constexpr bool kHold = CH <= 16;        // weights stay in registers
  extern __shared__ __align__(16) char smem[];
  __shared__ float parts[kGroups][2 * 2 * (TPR > 32 ? TPR / 32 : 1)];
  const int group = threadIdx.x / TPR, lane = threadIdx.x & 31;
  float* part = parts[group];
  char* xs = smem + threadIdx.x * Raw<Tx, VEC>::kBytes;
  char* us = smem + kDy + threadIdx.x * Raw<Tu, VEC>::kBytes;
  char* stats = smem + kStats + (threadIdx.x >> 5) * 8;    // of the warp: mean, rstd
  const int t = threadIdx.x % TPR;
  const int step = gridDim.x * kGroups;
  int row = blockIdx.x * kGroups + group;
  const auto fetch = [&](int r, int stage) {
    if (r < ntok) {
      const size_t base = static_cast<size_t>(r) * D;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (k * TPR + t) * VEC;
        if (c < D) {
          copy<VEC, kThreads>(xs + stage * kStage, k, x + base + c);
          copy<VEC, kThreads>(us + stage * kStage, k, dy + base + c);
        }
      }
      // one lane copies for its warp; a load here would hold up every row (0.100 ms instead of
      // 0.067 ms at 16384 x 4096 bf16)
      if (lane == 0) {
        copy_bytes<4>(stats + stage * kStage, mean + r);
        copy_bytes<4>(stats + stage * kStage + 4, rstd + r);
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
  float wv[kHold ? NV : 1][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * TPR + t) * VEC;
    if (kHold && c < D) weights(w, c, 1.f, wv[k]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[k][e] = db[k][e] = 0.f;
  }
  const float invD = 1.0f / D;
  int use = 0, fill = kStages - 1;
  for (int it = 0; row < ntok; ++it) {
    fetch(ahead(kStages - 1), fill);
    copies_wait<kStages - 1>();
    __syncwarp();
    const float2 st = *reinterpret_cast<const float2*>(stats + use * kStage);
    const float mu = st.x, rs = st.y;
    const char* xr = xs + use * kStage;
    const char* ur = us + use * kStage;
    float sum[2] = {0.f, 0.f};            // of n, and of n (x - mean)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (c < D) {
        float xv[VEC], uv[VEC], wl[VEC];
        unpack(staged<Tx, VEC, kThreads>(xr, k), xv);
        unpack(staged<Tu, VEC, kThreads>(ur, k), uv);
        if (!kHold) weights(w, c, 1.f, wl);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float n = uv[e] * (kHold ? wv[kHold ? k : 0][e] : wl[e]);
          sum[0] += n;
          sum[1] = fmaf(n, xv[e] - mu, sum[1]);
        }
      }
    }
    row_sum<TPR>(sum, part, it, group);
    const float m1 = -rs * sum[0] * invD, m2 = -rs * rs * sum[1] * invD;
    const size_t base = static_cast<size_t>(row) * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (c < D) {
        float xv[VEC], uv[VEC], wl[VEC], g[VEC];
        unpack(staged<Tx, VEC, kThreads>(xr, k), xv);
        unpack(staged<Tu, VEC, kThreads>(ur, k), uv);
        if (!kHold) weights(w, c, 1.f, wl);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (xv[e] - mu) * rs;
          dw[k][e] = fmaf(uv[e], xh, dw[k][e]);
          db[k][e] += uv[e];
          g[e] = fmaf(xh, m2, fmaf(uv[e] * (kHold ? wv[kHold ? k : 0][e] : wl[e]), rs, m1));
        }
        store(dx + base + c, g);
      }
    }
    __syncwarp();                         // the warp's statistics are read before their refill
    fill = use;
    use = use + 1 == kStages ? 0 : use + 1;
    row = ahead(1);
  }
  if (!partial) return;
  release_dependents();
  copies_wait<0>();
  float* mine = partial + static_cast<size_t>(blockIdx.x) * D;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * TPR + t) * VEC;
      if (c < D) {
        store(mine + c, dw[k]);
        store(mine + static_cast<size_t>(gridDim.x) * D + c, db[k]);
      }
    }
  } else {
    float* acc = reinterpret_cast<float*>(smem);
    float* own = acc + group * D;
    __syncthreads();                      // every group has read its rows from the ring
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * TPR + t) * VEC < D) store(own + (k * TPR + t) * VEC, dw[k]);
    write_partial<TPR>(acc, mine, D);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * TPR + t) * VEC < D) store(own + (k * TPR + t) * VEC, db[k]);
    write_partial<TPR>(acc, mine + static_cast<size_t>(gridDim.x) * D, D);
  }
}

// Any width: one channel at a time, bound like the forward's: 17 us at 4099 x 1001 bf16, 25 MB.
template <typename Tx, typename Tu, int TPR, int NV>
__global__ void __launch_bounds__(bwd_threads(TPR))
ln_bwd_any_kernel(const Tx* __restrict__ x, const Tu* __restrict__ dy,
                  const float* __restrict__ mean, const float* __restrict__ rstd,
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
      xv[k] = c < D ? Io<Tx>::ld(x, base + c) : mu;
      uv[k] = c < D ? Io<Tu>::ld(dy, base + c) : 0.f;
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
  release_dependents();
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

// Threads of a row and channels of each; D <= tpr * ch.
struct Shape {
  bool vec;
  int tpr, ch;
};

// Forward: a warp per row up to 1024 channels, otherwise a block with 32 channels per thread; few
// rows (at most two per SM) get more threads instead, since the row's own latency counts then.
Shape fwd_shape(int ntok, int D) {
  const bool few = ntok <= 2 * kSms;
  if (D % 8 == 0) {
    if (D <= 256) return {true, 32, 8};
    if (D <= 512) return {true, 32, 16};
    if (few && D <= 4096) return D <= 1024 ? Shape{true, 128, 8} : Shape{true, 512, 8};
    if (D <= 1024) return {true, 32, 32};
    if (D <= 2048) return {true, 128, 16};
    if (D <= 4096) return {true, 128, 32};
    if (D <= 8192) return {true, 256, 32};
    return {true, 512, 32};
  }
  if (D <= 256) return {false, 32, 8};
  if (D <= 1024) return {false, 128, 8};
  if (D <= 4096) return {false, 256, 16};
  return {false, 512, 32};
}
// Gradients: 16 channels per thread, of which three values each stay in registers; 32 where a
// block cannot be larger, and their weights are read again for every row.
Shape bwd_shape(int D) {
  if (D % 8 == 0) {
    if (D <= 256) return {true, 32, 8};
    int tpr = 32;
    while (tpr < 512 && tpr * 16 < D) tpr *= 2;
    return {true, tpr, tpr * 16 < D ? 32 : 16};
  }
  if (D <= 256) return {false, 32, 8};
  if (D <= 1024) return {false, 128, 8};
  if (D <= 4096) return {false, 256, 16};
  return {false, 512, 32};
}

template <int T, int N> struct Pick {
  static constexpr int tpr = T, ch = N;
};
template <typename F>
cudaError_t with_shape(const Shape& s, F&& f) {
  switch (s.tpr * 64 + s.ch) {
    case 32 * 64 + 8: return f(Pick<32, 8>{});
    case 32 * 64 + 16: return f(Pick<32, 16>{});
    case 32 * 64 + 32: return f(Pick<32, 32>{});
    case 64 * 64 + 16: return f(Pick<64, 16>{});
    case 128 * 64 + 8: return f(Pick<128, 8>{});
    case 128 * 64 + 16: return f(Pick<128, 16>{});
    case 128 * 64 + 32: return f(Pick<128, 32>{});
    case 256 * 64 + 16: return f(Pick<256, 16>{});
    case 256 * 64 + 32: return f(Pick<256, 32>{});
    case 512 * 64 + 8: return f(Pick<512, 8>{});
    case 512 * 64 + 16: return f(Pick<512, 16>{});
    case 512 * 64 + 32: return f(Pick<512, 32>{});
  }
  return cudaErrorInvalidConfiguration;
}
// Compiles only what a shape table can name.
constexpr bool fwd_vec(int tpr, int ch) {
  return tpr == 32 || tpr == 128 || (tpr == 256 && ch == 32) || (tpr == 512 && ch != 16);
}
constexpr bool bwd_vec(int tpr, int ch) {
  return ch == 16 || (tpr == 32 && ch == 8) || (tpr == 512 && ch == 32);
}
constexpr bool any_width(int tpr, int ch) {
  return (tpr == 32 && ch == 8) || (tpr == 128 && ch == 8) || (tpr == 256 && ch == 16) ||
         (tpr == 512 && ch == 32);
}

int bwd_blocks(const Shape& s, int ntok) {
  const int groups = bwd_threads(s.tpr) / s.tpr;
  const int per_sm = s.vec ? bwd_blocks_per_sm(s.tpr) : s.tpr > 256 ? 1 : 4;
  const long long need = (static_cast<long long>(ntok) + groups - 1) / groups;
  return need < kSms * per_sm ? static_cast<int>(need) : kSms * per_sm;
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
    constexpr int T = decltype(p)::tpr, N = decltype(p)::ch;
    if (!sh.vec) {
      if constexpr (any_width(T, N)) {
        return by_type(x_t, [&](auto tx) {
          using Tx = decltype(tx);
          ln_fwd_any_kernel<Tx, T, N><<<blocks, threads, 0, s>>>(
              static_cast<const Tx*>(x), w, b, eps, invD, AnyOut{y, y_t == DType::F32}, mean, rstd,
              ntok, D);
          return cudaGetLastError();
        });
      }
    } else if constexpr (fwd_vec(T, N)) {
      return by_type(x_t, [&](auto tx) {
        return by_type(y_t, [&](auto ty) {
          using Tx = decltype(tx);
          using Ty = decltype(ty);
          ln_fwd_kernel<Tx, Ty, T, N / kFwdVec><<<blocks, threads, 0, s>>>(
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
      constexpr int T = decltype(p)::tpr, N = decltype(p)::ch;
      constexpr int kThreads = bwd_threads(T);
      const size_t sums = kThreads / T > 1 ? static_cast<size_t>(kThreads / T) * D * sizeof(float) : 0;
      if (!sh.vec) {
        if constexpr (any_width(T, N)) {
          return by_type(x_t, [&](auto tx) {
            return by_type(dy_t, [&](auto tu) {
              using Tx = decltype(tx);
              using Tu = decltype(tu);
              const cudaError_t a = allow_smem(ln_bwd_any_kernel<Tx, Tu, T, N>, sums);
              if (a != cudaSuccess) return a;
              ln_bwd_any_kernel<Tx, Tu, T, N><<<blocks, kThreads, sums, s>>>(
                  static_cast<const Tx*>(x), static_cast<const Tu*>(dy), mean, rstd, w,
                  AnyOut{dx, dx_t == DType::F32}, part, ntok, D);
              return cudaGetLastError();
            });
          });
        }
      } else if constexpr (bwd_vec(T, N)) {
        return by_type(x_t, [&](auto tx) {
          return by_type(dy_t, [&](auto tu) {
            return by_type(dx_t, [&](auto tg) {
              using Tx = decltype(tx);
              using Tu = decltype(tu);
              using Tg = decltype(tg);
              const size_t ring =
                  static_cast<size_t>(bwd_stages<Tx, Tu>(T, N)) * bwd_stage_bytes<Tx, Tu>(T, N);
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
