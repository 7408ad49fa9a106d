// Gradients of the per-head GroupNorm + Swish gate (formulas in include/retention.h).
// Bound by HBM, then by instruction issue (75 %): o, g and d_y are read and d_o, d_g written once.
// Measured at 16384 x 16 x 512 bf16: 0.232 ms in a few graph replays (5.8 TB/s, 88 % of the measured
// copy rate), 0.263 ms in a loop of 3000 calls (78 %).  With a float32 o (8192 x 8 x 256, the rest bf16)
// 0.046 ms, 67 %: 38 us and the sum of the partial gradients, with 69 % of the issue slots used,
// since every tensor is then copied and stored in 8- or 16-byte vectors of four channels.
//
// A (token, head) row belongs to TPR threads (8 to 64, 16 channels each); up to a warp its sums
// are shuffles alone.  The threads stay with their head and walk the tokens: their channels' sums
// for d_weight and d_bias stay in registers, the weights in the L1 cache.  The next row is on
// its way to shared memory meanwhile.  The groups' sums go to the workspace and a second kernel
// adds them in a fixed order.
#include "norm_common.cuh"

namespace ret {
namespace {

using namespace norm;

constexpr int kThreads = 256;
// Blocks of an SM: 128 registers per thread.
constexpr int kBlocksPerSm = 2;
// Bytes of a stage (a row of o, g and d_y per group), and the stages (rows on their way, and one
// in use).  CH: channels of a thread.
template <typename To, typename Ti> constexpr int stage_bytes(int CH) {
  return kThreads * CH * static_cast<int>(sizeof(To) + 2 * sizeof(Ti));
}
template <typename To, typename Ti> constexpr int stage_count(int CH) {
  return stages(stage_bytes<To, Ti>(CH), kBlocksPerSm);
}

// swish(g) = g s and its derivative's factor s (1 + g (1 - s)), s = sigmoid(g)
// (the forms that take subnormals as zero; the others scale around them: 234 instead of 230 us)
__device__ __forceinline__ float sigmoid(float x) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}

template <typename To, typename Ti, typename Tg, int TPR, int CH>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
ng_bwd_kernel(const To* __restrict__ o, const Ti* __restrict__ g, const Ti* __restrict__ dy,
              const float* __restrict__ w, const float* __restrict__ b, float eps,
              Tg* __restrict__ d_o, Tg* __restrict__ d_g, float* __restrict__ partial, int ntok,
              int H, int dv, int lanes) {
  constexpr int VEC = vec_of<To, Ti, Tg>(), NV = CH / VEC;
  constexpr int kStages = stage_count<To, Ti>(CH), kStage = stage_bytes<To, Ti>(CH);
  constexpr int kG = kThreads * CH * static_cast<int>(sizeof(To));      // offsets in a stage
  constexpr int kDy = kG + kThreads * CH * static_cast<int>(sizeof(Ti));
  constexpr int kW = TPR > 32 ? TPR / 32 : 1;
  extern __shared__ __align__(16) char smem[];
  __shared__ float parts[kThreads / TPR][2 * kW * 4];
  char* os = smem + threadIdx.x * Raw<To, VEC>::kBytes;
  char* gs = smem + kG + threadIdx.x * Raw<Ti, VEC>::kBytes;
  char* us = smem + kDy + threadIdx.x * Raw<Ti, VEC>::kBytes;
  const int t = threadIdx.x % TPR, local = threadIdx.x / TPR;
  const int group = blockIdx.x * (kThreads / TPR) + local;
  const int head = group % H, first = group / H;      // first: token, and partial row
  const size_t token = static_cast<size_t>(H) * dv, stride = token * lanes;
  const int col = head * dv + t * VEC;                  // of the thread's first vector
  bool has[NV];                                       // groups of a warp may differ here
#pragma unroll
  for (int k = 0; k < NV; ++k) has[k] = first < lanes && (k * TPR + t) * VEC < dv;
  const auto fetch = [&](bool there, size_t at, int stage) {
    if (there) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (has[k]) {
          const size_t c = at + k * TPR * VEC;
          copy<VEC, kThreads>(os + stage * kStage, k, o + c);
          copy<VEC, kThreads>(gs + stage * kStage, k, g + c);
          copy<VEC, kThreads>(us + stage * kStage, k, dy + c);
        }
    }
    copies_commit();
  };
  size_t at = static_cast<size_t>(first) * token + col;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k)
    fetch(first + static_cast<long long>(k) * lanes < ntok, at + k * stride, k);
  float dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[k][e] = db[k][e] = 0.f;
  const float invD = 1.0f / dv;
  // all groups of a warp take the same number of turns (the sums are warp-wide shuffles)
  const int turns = static_cast<int>((static_cast<long long>(ntok) + lanes - 1) / lanes);
  int use = 0, fill = kStages - 1;
  long long n = first;
  for (int it = 0; it < turns; ++it) {
    const bool ok = n < ntok;
    fetch(n + static_cast<long long>(kStages - 1) * lanes < ntok, at + (kStages - 1) * stride, fill);
    copies_wait<kStages - 1>();
    float ov[NV][VEC], dt[NV][VEC], q[NV][VEC];
    float mean[1] = {0.f}, sum[3] = {0.f, 0.f, 0.f};   // sum: of (o - mu)^2, n and n (o - mu)
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ok && has[k]) {
        unpack(staged<To, VEC, kThreads>(os + use * kStage, k), ov[k]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) mean[0] += ov[k][e];
      }
    row_sum<TPR>(mean, parts[local], it, local);
    const float mu = mean[0] * invD;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ok && has[k]) {
        float gv[VEC], uv[VEC], wv[VEC];
        unpack(staged<Ti, VEC, kThreads>(gs + use * kStage, k), gv);
        unpack(staged<Ti, VEC, kThreads>(us + use * kStage, k), uv);
        weights(w, col + k * TPR * VEC, 1.f, wv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ov[k][e] -= mu;
          const float sg = sigmoid(gv[e]), us = uv[e] * sg;
          const float d = us * gv[e];                  // d_y swish(g)
          q[k][e] = us * fmaf(gv[e], 1.f - sg, 1.f);   // d_g / t
          dt[k][e] = d;
          sum[0] = fmaf(ov[k][e], ov[k][e], sum[0]);
          sum[1] = fmaf(d, wv[e], sum[1]);
          sum[2] = fmaf(d * wv[e], ov[k][e], sum[2]);
        }
      }
    row_sum<TPR>(sum, parts[local] + 2 * kW, it, local);
    const float rs = inv_std(sum[0] * invD, eps);
    const float m1 = -rs * sum[1] * invD, m2 = -rs * rs * sum[2] * invD;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ok && has[k]) {
        float go[VEC], gg[VEC], wv[VEC], bv[VEC];
        weights(w, col + k * TPR * VEC, 1.f, wv);
        weights(b, col + k * TPR * VEC, 0.f, bv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = ov[k][e] * rs;
          gg[e] = q[k][e] * fmaf(xh, wv[e], bv[e]);
          go[e] = fmaf(xh, m2, fmaf(dt[k][e] * wv[e], rs, m1));
          dw[k][e] = fmaf(dt[k][e], xh, dw[k][e]);
          db[k][e] += dt[k][e];
        }
        store(d_o + at + k * TPR * VEC, go);
        store(d_g + at + k * TPR * VEC, gg);
      }
    fill = use;
    use = use + 1 == kStages ? 0 : use + 1;
    n += lanes;
    at += stride;
  }
  if (!partial) return;
  release_dependents();
  float* mine = partial + static_cast<size_t>(first) * token + col;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (has[k]) {
      store(mine + k * TPR * VEC, dw[k]);
      store(mine + stride + k * TPR * VEC, db[k]);
    }
}

// Any width: a warp per row, one channel at a time.
template <typename To, typename Ti, int NV>
__global__ void __launch_bounds__(kThreads)
ng_bwd_any_kernel(const To* __restrict__ o, const Ti* __restrict__ g, const Ti* __restrict__ dy,
                  const float* __restrict__ w, const float* __restrict__ b, float eps,
                  AnyOut d_o, AnyOut d_g, float* __restrict__ partial, int ntok, int H,
                  int dv, int lanes) {
  const int t = threadIdx.x & 31;
  const int group = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int head = group % H, first = group / H;
  if (first >= lanes) return;
  const int c0 = head * dv;
  const size_t token = static_cast<size_t>(H) * dv;
  float dw[NV], db[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) dw[k] = db[k] = 0.f;
  const float invD = 1.0f / dv;
  for (long long n = first; n < ntok; n += lanes) {
    const size_t base = static_cast<size_t>(n) * token + c0;
    float ov[NV], gv[NV], uv[NV], mean[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = k * 32 + t;
      ov[k] = c < dv ? Io<To>::ld(o, base + c) : 0.f;
      gv[k] = c < dv ? Io<Ti>::ld(g, base + c) : 0.f;
      uv[k] = c < dv ? Io<Ti>::ld(dy, base + c) : 0.f;
      mean[0] += ov[k];
    }
    row_sum<32>(mean, nullptr, 0);
    const float mu = mean[0] * invD;
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = k * 32 + t;
      if (c < dv) {
        const float d = ov[k] - mu;
        const float m = uv[k] * (gv[k] * sigmoid(gv[k])) * (w ? w[c0 + c] : 1.f);
        sum[0] = fmaf(d, d, sum[0]);
        sum[1] += m;
        sum[2] = fmaf(m, d, sum[2]);
      }
    }
    row_sum<32>(sum, nullptr, 0);
    const float rs = inv_std(sum[0] * invD, eps);
    const float m1 = sum[1] * invD, m2 = sum[2] * invD * rs;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = k * 32 + t;
      if (c < dv) {
        const float sg = sigmoid(gv[k]), xh = (ov[k] - mu) * rs, us = uv[k] * sg, dt = us * gv[k];
        const float wc = w ? w[c0 + c] : 1.f, bc = b ? b[c0 + c] : 0.f;
        d_g.st(base + c, us * fmaf(xh, wc, bc) * fmaf(gv[k], 1.f - sg, 1.f));
        d_o.st(base + c, rs * (fmaf(dt, wc, -m1) - xh * m2));
        dw[k] = fmaf(dt, xh, dw[k]);
        db[k] += dt;
      }
    }
  }
  if (!partial) return;
  release_dependents();
  float* mine = partial + static_cast<size_t>(first) * token + c0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = k * 32 + t;
    if (c < dv) {
      mine[c] = dw[k];
      mine[static_cast<size_t>(lanes) * token + c] = db[k];
    }
  }
}

// Channels of a thread, and threads of a row.
int row_channels(int dv) { return dv > 64 ? 16 : 8; }
int row_threads(int dv) {
  if (dv % 8 != 0) return 32;
  int t = 8;
  while (t * row_channels(dv) < dv) t *= 2;
  return t;
}
// Token lanes: groups per head that are resident at once.
int token_lanes(int ntok, int H, int dv) {
  const long long groups = static_cast<long long>(kSms) * kBlocksPerSm * (kThreads / row_threads(dv));
  const long long per = groups / H > 1 ? groups / H : 1;
  return static_cast<int>(per < ntok ? per : ntok);
}

}  // namespace

int norm_gate_bwd_partial_rows(int ntok, int H, int dv) { return token_lanes(ntok, H, dv); }

cudaError_t launch_norm_gate_bwd(const void* o, DType o_t, const void* g, const void* dy,
                                 DType g_t, const float* w, const float* b, float eps, void* d_o,
                                 void* d_g, DType grad_t, float* dw, float* db, float* partial,
                                 int ntok, int H, int dv, cudaStream_t s) {
  const int lanes = token_lanes(ntok, H, dv), tpr = row_threads(dv);
  float* part = dw ? partial : nullptr;
  cudaError_t e = cudaSuccess;
  if (ntok > 0) {
    const long long groups = static_cast<long long>(lanes) * H;
    const int per = kThreads / tpr;
    const long long nb = (groups + per - 1) / per;
    if (nb > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const unsigned blocks = static_cast<unsigned>(nb);
    if (dv % 8 != 0) {
      const AnyOut go{d_o, grad_t == DType::F32}, gg{d_g, grad_t == DType::F32};
      e = by_type(o_t, [&](auto to) {
        return by_type(g_t, [&](auto ti) {
          using To = decltype(to);
          using Ti = decltype(ti);
          const auto run = [&](auto kern) {
            kern<<<blocks, kThreads, 0, s>>>(static_cast<const To*>(o), static_cast<const Ti*>(g),
                                             static_cast<const Ti*>(dy), w, b, eps, go, gg, part,
                                             ntok, H, dv, lanes);
            return cudaGetLastError();
          };
          if (dv <= 128) return run(ng_bwd_any_kernel<To, Ti, 4>);
          if (dv <= 256) return run(ng_bwd_any_kernel<To, Ti, 8>);
          return run(ng_bwd_any_kernel<To, Ti, 32>);
        });
      });
    } else {
      e = by_type(o_t, [&](auto to) {
        return by_type(g_t, [&](auto ti) {
          return by_type(grad_t, [&](auto tg) {
            using To = decltype(to);
            using Ti = decltype(ti);
            using Tg = decltype(tg);
            const auto run = [&](auto kern, int ch) {
              const size_t smem =
                  static_cast<size_t>(stage_count<To, Ti>(ch)) * stage_bytes<To, Ti>(ch);
              const cudaError_t a = allow_smem(kern, smem);
              if (a != cudaSuccess) return a;
              kern<<<blocks, kThreads, smem, s>>>(
                  static_cast<const To*>(o), static_cast<const Ti*>(g), static_cast<const Ti*>(dy),
                  w, b, eps, static_cast<Tg*>(d_o), static_cast<Tg*>(d_g), part, ntok, H, dv,
                  lanes);
              return cudaGetLastError();
            };
            if (row_channels(dv) == 8) return run(ng_bwd_kernel<To, Ti, Tg, 8, 8>, 8);
            if (tpr == 8) return run(ng_bwd_kernel<To, Ti, Tg, 8, 16>, 16);
            if (tpr == 16) return run(ng_bwd_kernel<To, Ti, Tg, 16, 16>, 16);
            if (tpr == 32) return run(ng_bwd_kernel<To, Ti, Tg, 32, 16>, 16);
            return run(ng_bwd_kernel<To, Ti, Tg, 64, 16>, 16);
          });
        });
      });
    }
  }
  if (e != cudaSuccess || !dw) return e;
  return sum_rows(partial, dw, db, lanes, H * dv, s);
}

}  // namespace ret
