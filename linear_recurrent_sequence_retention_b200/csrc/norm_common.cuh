// Shared by layer norm, its gradients and the gradients of the GroupNorm + gate:
// how a row is spread over threads, eight-element vectors, sums over a row's
// threads, per-thread copies into shared memory ahead of use, and the sum of the
// partial weight gradients.
//
// A row of D channels belongs to TPR threads; with VEC = 8 thread t of them holds
// the vectors t, t + TPR, ... (NV of them) of eight channels, with VEC = 1 (rows
// that do not divide into such vectors) the channels t, t + TPR, ...
#pragma once

#include "launch.h"

namespace ret {
namespace norm {

// ---- types -------------------------------------------------------------------

template <typename F>
cudaError_t by_type(DType t, F&& f) {
  return t == DType::F32 ? f(float{}) : f(__nv_bfloat16{});
}

// A tensor whose type is known at run time only (the VEC = 1 kernels).
struct Any {
  const void* p;
  bool f32;
  __device__ __forceinline__ float ld(size_t i) const {
    return f32 ? static_cast<const float*>(p)[i]
               : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
};
struct AnyOut {
  void* p;
  bool f32;
  __device__ __forceinline__ void st(size_t i, float v) const {
    if (f32)
      static_cast<float*>(p)[i] = v;
    else
      static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  }
};

// Eight consecutive elements as they are stored.
template <typename T> struct Raw8 {
  static constexpr int kU = static_cast<int>(sizeof(T)) / 2;     // 16-byte units
  uint4 u[kU];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int k = 0; k < Raw8<T>::kU; ++k) r.u[k] = __ldg(reinterpret_cast<const uint4*>(p) + k);
  return r;
}
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    v[4 * k] = __uint_as_float(r.u[k].x);
    v[4 * k + 1] = __uint_as_float(r.u[k].y);
    v[4 * k + 2] = __uint_as_float(r.u[k].z);
    v[4 * k + 3] = __uint_as_float(r.u[k].w);
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
// Eight weights; `none` where there are none.
__device__ __forceinline__ void weights8(const float* w, int c, float none, float (&v)[8]) {
  if (w) {
    unpack(load8(w + c), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = none;
  }
}

// 1 / sqrt(var + eps), to two units of the last place: a row's one reciprocal root costs every
// thread of the row, and the correctly rounded square root and division take ~40 instructions.
__device__ __forceinline__ float inv_std(float var, float eps) { return rsqrtf(var + eps); }

// ---- sums over the TPR threads of a row ----------------------------------------

// Every thread gets the sums of the N values.  Rows of more than a warp meet in
// `part` (the row's own two buffers of warps x N, by the parity of `turn`: one barrier of the
// row's threads per sum; `group` numbers the rows of a block).
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* part, int turn, int group = 0) {
#pragma unroll
  for (int off = (TPR < 32 ? TPR : 32) / 2; off; off >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if constexpr (TPR > 32) {
    constexpr int kW = TPR / 32;
    float* p = part + (turn & 1) * kW * N;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) p[(threadIdx.x % TPR / 32) * N + k] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
    // every kW lanes read the warps' sums and add them in the same tree
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = p[(threadIdx.x % kW) * N + k];
#pragma unroll
    for (int off = kW / 2; off; off >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  }
}

// ---- copies ahead of use ---------------------------------------------------------

// Every thread copies the vectors that it will read itself, so the only wait is for its own
// copies.  Unit n of thread t lies at [n][t]: no bank conflicts.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Stages of `bytes` each that fit where `blocks` blocks share an SM: at most four.
constexpr int stages(int bytes, int blocks) {
  const int fit = (220 * 1024 / blocks) / bytes;
  return fit > 4 ? 4 : fit < 1 ? 1 : fit;
}
template <typename T>
__device__ __forceinline__ void copy8(uint4* slot, int threads, const T* src) {
#pragma unroll
  for (int k = 0; k < Raw8<T>::kU; ++k)
    copy16(slot + k * threads, reinterpret_cast<const uint4*>(src) + k);
}
template <typename T>
__device__ __forceinline__ Raw8<T> read8(const uint4* slot, int threads) {
  Raw8<T> r;
#pragma unroll
  for (int k = 0; k < Raw8<T>::kU; ++k) r.u[k] = slot[k * threads];
  return r;
}

// ---- sum of partial rows ---------------------------------------------------------

// out[j][c] = sum over rows of part[j][row][c], j = 0, 1: eight row groups, each in order, then
// the groups in order.
static __global__ void __launch_bounds__(256)
sum_rows_kernel(const float* __restrict__ part, float* __restrict__ out0, float* __restrict__ out1,
                int rows, int width) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* p = part + static_cast<size_t>(blockIdx.y) * rows * width;
  float v = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int r = g; r < rows; r += 8) v += p[static_cast<size_t>(r) * width + c];
  }
  s[g][lane] = v;
  __syncthreads();
  if (g > 0 || c >= width) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) v += s[k][lane];
  (blockIdx.y ? out1 : out0)[c] = v;
}
inline cudaError_t sum_rows(const float* part, float* out0, float* out1, int rows, int width,
                            cudaStream_t s) {
  sum_rows_kernel<<<dim3((width + 31) / 32, 2), 256, 0, s>>>(part, out0, out1, rows, width);
  return cudaGetLastError();
}

constexpr int kSms = 148;

template <typename K>
cudaError_t allow_smem(K* kern, size_t bytes) {
  return bytes <= 32 * 1024         // the rest of the default 48 KB is for static shared memory
             ? cudaSuccess
             : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(bytes));
}

}  // namespace norm
}  // namespace ret
