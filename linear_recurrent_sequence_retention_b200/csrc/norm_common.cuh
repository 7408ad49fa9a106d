// Shared by layer norm, its gradients and the gradients of the GroupNorm + gate:
// how a row is spread over threads, vectors, sums over a row's
// threads, per-thread copies into shared memory ahead of use, and the sum of the
// partial weight gradients.
//
// A row of D channels belongs to TPR threads; thread t of them holds the vectors t, t + TPR,
// ... (NV of them) of VEC channels.  A vector is at most 16 bytes of any tensor, so that the
// threads of a warp touch whole sectors with every access: VEC = 8 where all tensors are bf16,
// 4 where one is float32 (with 32-byte vectors every sector is fetched twice: the gradients of a
// float32 layer norm at 4096 x 4096 took 0.054 ms that way).  VEC = 1 serves rows that do not
// divide by eight.
#pragma once

#include "launch.h"

namespace ret {
namespace norm {

// ---- types -------------------------------------------------------------------

template <typename F>
cudaError_t by_type(DType t, F&& f) {
  return t == DType::F32 ? f(float{}) : f(__nv_bfloat16{});
}

// Outputs of the VEC = 1 kernels: the type is looked up per element.  (Their inputs are typed:
// loads behind a branch wait for one another, 0.028 ms instead of 0.008 ms at 4099 x 1001.)
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

// VEC consecutive elements as they are stored: 8 or 16 bytes.
template <typename T, int VEC> struct Raw {
  static constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
  static constexpr int kWords = kBytes / 4;
  static_assert(kBytes == 8 || kBytes == 16, "one access");
  uint32_t w[kWords];
};
template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&w)[WORDS], const void* p) {
  if constexpr (WORDS == 4) {
    const uint4 v = *static_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *static_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}
template <int VEC, typename T>
__device__ __forceinline__ Raw<T, VEC> load(const T* p) {
  Raw<T, VEC> r;
  load_words(r.w, p);
  return r;
}
template <int VEC>
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, VEC>& r, float (&v)[VEC]) {
#pragma unroll
  for (int k = 0; k < VEC / 2; ++k) {
    v[2 * k] = __uint_as_float(r.w[k] << 16);
    v[2 * k + 1] = __uint_as_float(r.w[k] & 0xffff0000u);
  }
}
template <int VEC>
__device__ __forceinline__ void unpack(const Raw<float, VEC>& r, float (&v)[VEC]) {
#pragma unroll
  for (int k = 0; k < VEC; ++k) v[k] = __uint_as_float(r.w[k]);
}
template <int VEC>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[VEC]) {
  uint32_t w[VEC / 2];
#pragma unroll
  for (int k = 0; k < VEC / 2; ++k) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int VEC>
__device__ __forceinline__ void store(float* p, const float (&v)[VEC]) {
#pragma unroll
  for (int k = 0; k < VEC; k += 4)
    *reinterpret_cast<float4*>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
}
// VEC weights; `none` where there are none.
template <int VEC>
__device__ __forceinline__ void weights(const float* w, int c, float none, float (&v)[VEC]) {
#pragma unroll
  for (int k = 0; k < VEC; k += 4) {
    const float4 f = w ? __ldg(reinterpret_cast<const float4*>(w + c + k))
                       : make_float4(none, none, none, none);
    v[k] = f.x, v[k + 1] = f.y, v[k + 2] = f.z, v[k + 3] = f.w;
  }
}
// 8 where every tensor is bf16, else 4.
template <typename... T> constexpr int vec_of() {
  return ((sizeof(T) == 2) && ...) ? 8 : 4;
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
// copies.  Vector n of thread t lies at [n][t]: no bank conflicts.
template <int BYTES>
__device__ __forceinline__ void copy_bytes(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Stages of `bytes` each: the row in use and the next, where they fit for `blocks` blocks of an SM.
// (Three and four stages were slower: norm-gate gradients at 16384 x 16 x 512 bf16 0.246 and 0.253 ms
// instead of 0.236 ms.  The weights live in what shared memory leaves of the L1 cache.)
constexpr int stages(int bytes, int blocks) {
  return 2 * bytes <= 216 * 1024 / blocks ? 2 : 1;
}
// `slot`: the thread's place in the first vector of a tensor's part of a stage.
template <int VEC, int THREADS, typename T>
__device__ __forceinline__ void copy(char* slot, int n, const T* src) {
  copy_bytes<Raw<T, VEC>::kBytes>(slot + n * (THREADS * Raw<T, VEC>::kBytes), src);
}
template <typename T, int VEC, int THREADS>
__device__ __forceinline__ Raw<T, VEC> staged(const char* slot, int n) {
  Raw<T, VEC> r;
  load_words(r.w, slot + n * (THREADS * Raw<T, VEC>::kBytes));
  return r;
}

// ---- sum of partial rows ---------------------------------------------------------

// Lets the dependent kernel below start setting up; it still waits for the whole of this grid.
__device__ __forceinline__ void release_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// out[j][c] = sum over rows of part[j][row][c], j = 0, 1: 32 row groups, each in order, then
// the groups in order.  Launched so that its start overlaps the end of the kernel that
// writes `part`.
constexpr int kRowGroups = 32;
static __global__ void __launch_bounds__(32 * kRowGroups)
sum_rows_kernel(const float* __restrict__ part, float* __restrict__ out0, float* __restrict__ out1,
                int rows, int width) {
  __shared__ float s[kRowGroups][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* p = part + static_cast<size_t>(blockIdx.y) * rows * width;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int r = g; r < rows; r += kRowGroups) v += __ldcg(p + static_cast<size_t>(r) * width + c);
  }
  s[g][lane] = v;
  __syncthreads();
  if (g > 0 || c >= width) return;
#pragma unroll
  for (int k = 1; k < kRowGroups; ++k) v += s[k][lane];
  (blockIdx.y ? out1 : out0)[c] = v;
}
inline cudaError_t sum_rows(const float* part, float* out0, float* out1, int rows, int width,
                            cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((width + 31) / 32, 2);
  cfg.blockDim = dim3(32 * kRowGroups);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sum_rows_kernel, part, out0, out1, rows, width);
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
