// Gated linear recurrence (ql.gl blog on Griffin/Hawk, section "Hawk"):
//     h_t = a_t h_(t-1) + b_t x_t, element by element, with
//     s = sigmoid(r), y = c softplus(lam) s, a = exp(-y), b = sqrt(1 - a^2) sigmoid(i),
// its gradients, and the one-token step.
//
// A token is the affine map h -> a h + v (v = b x), and a run of tokens is one
// too: (A, V) then (a, v) is (a A, a V + v).  So time is split: a CTA takes 64
// channels and 64 tokens, a warp 8 of those tokens, and a cluster of S CTAs 64 S
// consecutive tokens per round.  Every warp forms the map of its 8 tokens from
// registers, the maps of the CTA's 8 warps meet in shared memory and those of
// the cluster's CTAs through distributed shared memory (one cluster barrier per
// round); each warp then applies its tokens to the state that enters them.
// Every input is read from HBM once and every output written once.  The
// gradients run the same scheme from the last round to the first on
// e -> a (dh + e), with the forward's states formed again from the state that
// enters each 64-token tile, which the forward stored.
//
// The inputs of the next round are copied to shared memory (cp.async) while the
// current one is computed.
#include <type_traits>

#include "launch.h"
#include "tc_ptx.cuh"

namespace ret {
namespace {

constexpr int kTile = kGlrChunk;    // tokens of a CTA per round
constexpr int kWarps = 8;
constexpr int kRun = kTile / kWarps;   // tokens of a warp
constexpr int kChan = 64;           // channels of a CTA: two per lane
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSplit = 16;       // CTAs of a cluster

// How a lane's two channels lie and how rows reach shared memory.
//   kWide: channels 2l, 2l+1; rows are copied in 16-byte pieces (D e bytes divide by 16)
//   kEven: channels 2l, 2l+1; 4-byte pieces (D even)
//   kOdd:  channels l, l+32; float32 in 4-byte pieces, bf16 read straight from global
//          memory (its rows start at odd multiples of two bytes)
enum { kWide = 0, kEven = 1, kOdd = 2 };

// ---- gates -----------------------------------------------------------------

__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid(float x) {
  return rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * x));
}

// a = exp(-y) and root = sqrt(1 - a^2) for y >= 0, both to a few units of their
// own last place: -y = n ln 2 + f, |f| <= ln 2 / 2, and with p = e^f - 1 (Taylor;
// the eighth term is below 2^-25 of the first) a = 2^n p + 2^n and
// 1 - a = 1 - 2^n - 2^n p, so 1 - a^2 = (1 - a)(1 + a) cancels nothing for decays
// near one.  Above y = 87 a counts as zero (it is below 1.7e-38); below the
// normal range of 1 - a^2 root is zero.
__device__ __forceinline__ void decay(float y, float& a, float& root) {
  constexpr float kMagic = 12582912.f;           // 1.5 * 2^23: adding it rounds to an integer
  const bool gone = y > 87.f;                    // NaN stays
  y = gone ? 87.f : y;
  const float m = fmaf(y, -1.4426950408889634f, kMagic);
  const float n = m - kMagic;
  float f = fmaf(n, -0.693147182464599609375f, -y);   // ln 2 in two parts
  f = fmaf(n, 1.904654290582768e-9f, f);
  float p = fmaf(f, 1.f / 5040.f, 1.f / 720.f);
  p = fmaf(f, p, 1.f / 120.f);
  p = fmaf(f, p, 1.f / 24.f);
  p = fmaf(f, p, 1.f / 6.f);
  p = fmaf(f, p, 0.5f);
  p = fmaf(f * f, p, f);
  const float s = gone ? 0.f : __int_as_float((__float_as_int(m) << 23) + 0x3f800000);   // 2^n
  a = fmaf(s, p, s);
  const float below = fmaf(-s, p, 1.f - s);      // 1 - a
  const float z = fmaf(below, a, below);
  root = z < 1.2e-38f ? 0.f : z * rsqrt_approx(z);
}

// ---- sequences and tiles ---------------------------------------------------

// First chunk row of sequence s, which starts at flat token n.
__device__ __forceinline__ long long chunk_row(int n, int s) { return n / kGlrChunk + s; }

// Reports offsets that are not 0 = cu[0] <= .. <= cu[nseq] = Ttot.
__device__ __forceinline__ void check_offsets(const SeqLayout& L, int s, unsigned* err) {
  if (L.cu == nullptr) return;
  const int a = L.cu[s], b = L.cu[s + 1];
  if ((s == 0 && a != 0) || b < a || (s == L.nseq - 1 && b != L.Ttot))
    raise_error(err, kErrDeviceData);
}

struct Args {
  const void* x;
  const void* r;
  const void* i;
  const float* lam;
  float c;
  SeqLayout L;
  int D, groups, split;      // split: CTAs per cluster
  unsigned* err;
};

template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T> constexpr int row_bytes() { return kChan * static_cast<int>(sizeof(T)); }
template <typename T, int MODE> constexpr bool staged() { return MODE != kOdd || sizeof(T) == 4; }

// Copies a warp's rows t .. t+7 (those below t1), channels c0 .. c0+63, to `dst`.
template <typename T, int MODE>
__device__ __forceinline__ void stage_rows(char* dst, const T* src, int t, int t1, int c0, int D,
                                           int lane) {
  if constexpr (staged<T, MODE>()) {
    constexpr int kPiece = MODE == kWide ? 16 : 4;
    constexpr int kPer = row_bytes<T>() / kPiece;       // pieces of a row
    constexpr int kElems = kPiece / static_cast<int>(sizeof(T));
    const uint32_t d = tc::smem_u32(dst);
#pragma unroll
    for (int k = 0; k < kRun * kPer / 32; ++k) {
      const int idx = k * 32 + lane, row = idx / kPer, p = idx % kPer;
      if (t + row < t1 && c0 + p * kElems < D)
        cp_async<kPiece>(d + row * row_bytes<T>() + p * kPiece,
                         src + static_cast<size_t>(t + row) * D + c0 + p * kElems);
    }
  }
}

// A lane's two channels of row k: from shared memory, or (kOdd bf16) from global.
template <typename T, int MODE>
__device__ __forceinline__ float2 row_pair(const char* st, const T* src, int k, int t, bool okt,
                                           int cA, int cB, int D, int lane) {
  if constexpr (!staged<T, MODE>()) {
    const size_t at = static_cast<size_t>(t) * D;
    float2 v = make_float2(0.f, 0.f);
    if (okt && cA < D) v.x = Io<T>::ld(src, at + cA);
    if (okt && cB < D) v.y = Io<T>::ld(src, at + cB);
    return v;
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(st + k * row_bytes<T>() + lane * 4);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  } else if constexpr (MODE == kOdd) {
    const float* p = reinterpret_cast<const float*>(st + k * row_bytes<T>());
    return make_float2(p[lane], p[lane + 32]);
  } else {
    return *reinterpret_cast<const float2*>(st + k * row_bytes<T>() + lane * 8);
  }
}

template <typename T, int MODE>
__device__ __forceinline__ void store_pair(T* dst, int t, float2 v, int cA, int cB, int D) {
  const size_t at = static_cast<size_t>(t) * D;
  if constexpr (MODE == kOdd) {
    if (cA < D) Io<T>::st(dst, at + cA, v.x);
    if (cB < D) Io<T>::st(dst, at + cB, v.y);
  } else if (cA < D) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + at + cA) = __floats2bfloat162_rn(v.x, v.y);
    else
      *reinterpret_cast<float2*>(dst + at + cA) = v;
  }
}

__device__ __forceinline__ float2 load2(const float* p, size_t at, int cA, int cB, int D) {
  return make_float2(p && cA < D ? p[at + cA] : 0.f, p && cB < D ? p[at + cB] : 0.f);
}
__device__ __forceinline__ void store2(float* p, size_t at, float2 v, int cA, int cB, int D) {
  if (cA < D) p[at + cA] = v.x;
  if (cB < D) p[at + cB] = v.y;
}

__device__ __forceinline__ void st_cluster_f32x4(uint32_t remote, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(remote), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// Affine maps of a lane's two channels: (A.x, V.x, A.y, V.y).
__device__ __forceinline__ float2 apply(const float4& m, float2 h) {
  return make_float2(fmaf(m.x, h.x, m.y), fmaf(m.z, h.y, m.w));
}
// first m, then n
__device__ __forceinline__ float4 then(const float4& m, const float4& n) {
  return make_float4(n.x * m.x, fmaf(n.x, m.y, n.y), n.z * m.z, fmaf(n.z, m.w, n.w));
}

// Maps exchanged in a round, double-buffered by the round's parity: a buffer is
// written again two rounds later, and every reader has passed the barrier of
// the round between by then.
using Maps = float4[32];             // one map per lane

__host__ __device__ constexpr size_t warp_maps_bytes() { return 2 * kWarps * sizeof(Maps); }
__host__ __device__ constexpr size_t cta_maps_bytes(int split) {
  return split > 1 ? 2 * split * sizeof(Maps) : 0;
}

// ---- forward ---------------------------------------------------------------

template <typename Ti, typename Th, int MODE>
__global__ void __launch_bounds__(kThreads)
glr_fwd_kernel(Args p, const float* __restrict__ state_in, float* __restrict__ state_out,
               Th* __restrict__ h, float* __restrict__ chunk_states) {
  extern __shared__ __align__(16) char smem[];
  constexpr int kArray = kRun * row_bytes<Ti>();        // a warp's rows of one input
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = p.split;
  Maps* warp_maps = reinterpret_cast<Maps*>(smem);                       // [2][kWarps]
  Maps* cta_maps = reinterpret_cast<Maps*>(smem + warp_maps_bytes());    // [2][S]
  char* ring = smem + warp_maps_bytes() + cta_maps_bytes(S) + warp * (2 * 3 * kArray);
  const int rank = static_cast<int>(blockIdx.x % S);
  const int pair = static_cast<int>(blockIdx.x / S);
  const int seq = pair / p.groups, c0 = (pair % p.groups) * kChan;
  const int D = p.D;
  const int cA = c0 + (MODE == kOdd ? lane : 2 * lane), cB = MODE == kOdd ? cA + 32 : cA + 1;
  const Ti* x = static_cast<const Ti*>(p.x);
  const Ti* r = static_cast<const Ti*>(p.r);
  const Ti* i = static_cast<const Ti*>(p.i);
  int t0, t1;
  seq_bounds(p.L, seq, t0, t1);
  if (c0 == 0 && rank == 0 && threadIdx.x == 0) check_offsets(p.L, seq, p.err);
  const int rounds = ceil_div(t1 - t0, kTile * S);
  const auto first = [&](int j) { return t0 + ((j * S + rank) * kWarps + warp) * kRun; };
  const auto fetch = [&](int j) {
    char* st = ring + (j & 1) * 3 * kArray;
    if (j < rounds) {
      stage_rows<Ti, MODE>(st, x, first(j), t1, c0, D, lane);
      stage_rows<Ti, MODE>(st + kArray, r, first(j), t1, c0, D, lane);
      stage_rows<Ti, MODE>(st + 2 * kArray, i, first(j), t1, c0, D, lane);
    }
    cp_commit();
  };
  fetch(0);
  const float2 lm = load2(p.lam, 0, cA, cB, D);
  const float2 ysc = make_float2(p.c * softplus(lm.x), p.c * softplus(lm.y));
  float2 carry = load2(state_in, static_cast<size_t>(seq) * D, cA, cB, D);
  if (S > 1) tc::cluster_sync();       // every CTA of the cluster runs before its memory is written
  for (int j = 0; j < rounds; ++j) {
    fetch(j + 1);
    cp_wait<1>();
    __syncwarp();
    const char* st = ring + (j & 1) * 3 * kArray;
    const int t = first(j);
    float2 a[kRun], v[kRun];
    float4 m = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const bool ok = t + k < t1;
      const float2 xv = row_pair<Ti, MODE>(st, x, k, t + k, ok, cA, cB, D, lane);
      const float2 rv = row_pair<Ti, MODE>(st + kArray, r, k, t + k, ok, cA, cB, D, lane);
      const float2 iv = row_pair<Ti, MODE>(st + 2 * kArray, i, k, t + k, ok, cA, cB, D, lane);
      float2 root;
      decay(ysc.x * sigmoid(rv.x), a[k].x, root.x);
      decay(ysc.y * sigmoid(rv.y), a[k].y, root.y);
      v[k] = make_float2(root.x * sigmoid(iv.x) * xv.x, root.y * sigmoid(iv.y) * xv.y);
      if (!ok) {                          // the identity
        a[k] = make_float2(1.f, 1.f);
        v[k] = make_float2(0.f, 0.f);
      }
      m = then(m, make_float4(a[k].x, v[k].x, a[k].y, v[k].y));
    }
    Maps* wm = warp_maps + (j & 1) * kWarps;
    wm[warp][lane] = m;
    __syncthreads();
    float4 before = make_float4(1.f, 0.f, 1.f, 0.f), total = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) before = total;
      total = then(total, wm[w][lane]);
    }
    float2 enter = carry;
    if (S > 1) {
      Maps* cm = cta_maps + (j & 1) * S;
      for (int q = warp; q < S; q += kWarps)
        st_cluster_f32x4(tc::cluster_addr(&cm[rank][lane], q), total);
      tc::cluster_sync();
      for (int q = 0; q < S; ++q) {
        if (q == rank) enter = carry;
        carry = apply(cm[q][lane], carry);
      }
    } else {
      carry = apply(total, carry);
    }
    const int tile = j * S + rank;
    if (chunk_states && warp == 0 && t < t1)
      store2(chunk_states, static_cast<size_t>(chunk_row(t0, seq) + tile) * D, enter, cA, cB, D);
    float2 hs = apply(before, enter);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      hs = make_float2(fmaf(a[k].x, hs.x, v[k].x), fmaf(a[k].y, hs.y, v[k].y));
      if (t + k < t1) store_pair<Th, MODE>(h, t + k, hs, cA, cB, D);
    }
  }
  if (state_out && rank == 0 && warp == 0)
    store2(state_out, static_cast<size_t>(seq) * D, carry, cA, cB, D);
}

// ---- gradients -------------------------------------------------------------

template <typename Ti, typename Tu, typename Tg, int MODE>
__global__ void __launch_bounds__(kThreads)
glr_bwd_kernel(Args p, const float* __restrict__ chunk_states, const Tu* __restrict__ dh,
               const float* __restrict__ d_state_out, Tg* __restrict__ dx, Tg* __restrict__ dr,
               Tg* __restrict__ di, float* __restrict__ d_state_in, float* __restrict__ partial) {
  extern __shared__ __align__(16) char smem[];
  constexpr int kArray = kRun * row_bytes<Ti>(), kUp = kRun * row_bytes<Tu>();
  constexpr int kStage = 3 * kArray + kUp;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = p.split;
  Maps* warp_maps = reinterpret_cast<Maps*>(smem);                       // [2][kWarps]
  Maps* cta_maps = reinterpret_cast<Maps*>(smem + warp_maps_bytes());    // [2][S]
  float2(*wf)[kWarps][32] = reinterpret_cast<float2(*)[kWarps][32]>(
      smem + warp_maps_bytes() + cta_maps_bytes(S));
  char* ring = reinterpret_cast<char*>(wf + 2) + warp * (2 * kStage);
  const int rank = static_cast<int>(blockIdx.x % S);
  const int pair = static_cast<int>(blockIdx.x / S);
  const int seq = pair / p.groups, c0 = (pair % p.groups) * kChan;
  const int D = p.D;
  const int cA = c0 + (MODE == kOdd ? lane : 2 * lane), cB = MODE == kOdd ? cA + 32 : cA + 1;
  const Ti* x = static_cast<const Ti*>(p.x);
  const Ti* r = static_cast<const Ti*>(p.r);
  const Ti* i = static_cast<const Ti*>(p.i);
  int t0, t1;
  seq_bounds(p.L, seq, t0, t1);
  if (c0 == 0 && rank == 0 && threadIdx.x == 0) check_offsets(p.L, seq, p.err);
  const int rounds = ceil_div(t1 - t0, kTile * S);
  const auto first = [&](int j) { return t0 + ((j * S + rank) * kWarps + warp) * kRun; };
  const auto fetch = [&](int j) {
    char* st = ring + (j & 1) * kStage;
    if (j >= 0) {
      stage_rows<Ti, MODE>(st, x, first(j), t1, c0, D, lane);
      stage_rows<Ti, MODE>(st + kArray, r, first(j), t1, c0, D, lane);
      stage_rows<Ti, MODE>(st + 2 * kArray, i, first(j), t1, c0, D, lane);
      stage_rows<Tu, MODE>(st + 3 * kArray, dh, first(j), t1, c0, D, lane);
    }
    cp_commit();
  };
  const auto entering = [&](int j) {
    const int tile = j * S + rank;
    if (j < 0 || t0 + tile * kTile >= t1) return make_float2(0.f, 0.f);
    return load2(chunk_states, static_cast<size_t>(chunk_row(t0, seq) + tile) * D, cA, cB, D);
  };
  fetch(rounds - 1);
  float2 cs = entering(rounds - 1);
  const float2 lm = load2(p.lam, 0, cA, cB, D);
  const float2 ysc = make_float2(p.c * softplus(lm.x), p.c * softplus(lm.y));
  const size_t so = static_cast<size_t>(seq) * D;
  float2 carry = load2(d_state_out, so, cA, cB, D);
  float2 usum = make_float2(0.f, 0.f);
  if (S > 1) tc::cluster_sync();
  for (int j = rounds - 1; j >= 0; --j) {
    __syncwarp();                         // the buffer refilled now was read to the round's end
    fetch(j - 1);
    const float2 cs_next = entering(j - 1);
    cp_wait<1>();
    __syncwarp();
    const char* st = ring + (j & 1) * kStage;
    const int t = first(j);
    // the run's map of h forwards (product in fw, sum below) and of e backwards
    float2 a[kRun], root[kRun], sr[kRun], si[kRun];
    float4 fw = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const bool ok = t + k < t1;
      const float2 xv = row_pair<Ti, MODE>(st, x, k, t + k, ok, cA, cB, D, lane);
      const float2 rv = row_pair<Ti, MODE>(st + kArray, r, k, t + k, ok, cA, cB, D, lane);
      const float2 iv = row_pair<Ti, MODE>(st + 2 * kArray, i, k, t + k, ok, cA, cB, D, lane);
      sr[k] = make_float2(sigmoid(rv.x), sigmoid(rv.y));
      si[k] = make_float2(sigmoid(iv.x), sigmoid(iv.y));
      decay(ysc.x * sr[k].x, a[k].x, root[k].x);
      decay(ysc.y * sr[k].y, a[k].y, root[k].y);
      float2 v = make_float2(root[k].x * si[k].x * xv.x, root[k].y * si[k].y * xv.y);
      if (!ok) {                          // the identity
        a[k] = make_float2(1.f, 1.f);
        v = make_float2(0.f, 0.f);
      }
      fw = then(fw, make_float4(a[k].x, v.x, a[k].y, v.y));
    }
    float2 w = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = kRun - 1; k >= 0; --k) {
      const bool ok = t + k < t1;
      const float2 u = row_pair<Tu, MODE>(st + 3 * kArray, dh, k, t + k, ok, cA, cB, D, lane);
      if (ok)
        w = make_float2(a[k].x * (u.x + w.x), a[k].y * (u.y + w.y));
    }
    Maps* wm = warp_maps + (j & 1) * kWarps;
    wm[warp][lane] = make_float4(fw.x, w.x, fw.z, w.y);
    wf[j & 1][warp][lane] = make_float2(fw.y, fw.w);
    __syncthreads();
    float2 hs = cs;                       // the state that enters this warp's run
    for (int q = 0; q < warp; ++q) {
      const float4 mq = wm[q][lane];
      const float2 vq = wf[j & 1][q][lane];
      hs = make_float2(fmaf(mq.x, hs.x, vq.x), fmaf(mq.z, hs.y, vq.y));
    }
    float4 after = make_float4(1.f, 0.f, 1.f, 0.f), total = after;
#pragma unroll
    for (int q = kWarps - 1; q >= 0; --q) {
      if (q == warp) after = total;
      total = then(total, wm[q][lane]);
    }
    float2 e = carry;
    if (S > 1) {
      Maps* cm = cta_maps + (j & 1) * S;
      for (int q = warp; q < S; q += kWarps)
        st_cluster_f32x4(tc::cluster_addr(&cm[rank][lane], q), total);
      tc::cluster_sync();
      for (int q = S - 1; q >= 0; --q) {
        if (q == rank) e = carry;
        carry = apply(cm[q][lane], carry);
      }
    } else {
      carry = apply(total, carry);
    }
    e = apply(after, e);
    float2 hp[kRun];                      // the state before each token
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      hp[k] = hs;
      const bool ok = t + k < t1;
      const float2 xv = row_pair<Ti, MODE>(st, x, k, t + k, ok, cA, cB, D, lane);
      if (ok)
        hs = make_float2(fmaf(a[k].x, hs.x, root[k].x * si[k].x * xv.x),
                         fmaf(a[k].y, hs.y, root[k].y * si[k].y * xv.y));
    }
#pragma unroll
    for (int k = kRun - 1; k >= 0; --k) {
      const bool ok = t + k < t1;
      if (!ok) continue;
      const float2 xv = row_pair<Ti, MODE>(st, x, k, t + k, ok, cA, cB, D, lane);
      const float2 uv = row_pair<Tu, MODE>(st + 3 * kArray, dh, k, t + k, ok, cA, cB, D, lane);
      float2 gx, gi, gr;
      const auto one = [](float a, float root, float sr, float si, float ysc, float x, float dh,
                          float hp, float& e, float& usum, float& gx, float& gr, float& gi) {
        const float G = dh + e, inv = root > 0.f ? rcp_approx(root) : 0.f;
        gx = G * (root * si);
        gi = gx * x * (1.f - si);
        const float u = G * a * (ysc * sr) * fmaf(a * inv, si * x, -hp);
        gr = u * (1.f - sr);
        usum += u;
        e = a * G;
      };
      one(a[k].x, root[k].x, sr[k].x, si[k].x, ysc.x, xv.x, uv.x, hp[k].x, e.x, usum.x, gx.x, gr.x,
          gi.x);
      one(a[k].y, root[k].y, sr[k].y, si[k].y, ysc.y, xv.y, uv.y, hp[k].y, e.y, usum.y, gx.y, gr.y,
          gi.y);
      store_pair<Tg, MODE>(dx, t + k, gx, cA, cB, D);
      store_pair<Tg, MODE>(dr, t + k, gr, cA, cB, D);
      store_pair<Tg, MODE>(di, t + k, gi, cA, cB, D);
    }
    cs = cs_next;
  }
  if (d_state_in && rank == 0 && warp == 0) store2(d_state_in, so, carry, cA, cB, D);
  // this CTA's part of sum u, its warps in order
  __syncthreads();
  wf[0][warp][lane] = usum;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int q = 1; q < kWarps; ++q) {
      usum.x += wf[0][q][lane].x;
      usum.y += wf[0][q][lane].y;
    }
    store2(partial, (static_cast<size_t>(seq) * S + rank) * D, usum, cA, cB, D);
  }
}

// d_lam = (sum of the partial rows) sigmoid(lam) / softplus(lam).  32 channels
// per block; eight row groups, each in order, then the groups in order.
__global__ void __launch_bounds__(256)
glr_dlam_kernel(const float* __restrict__ partial, const float* __restrict__ lam,
                float* __restrict__ d_lam, long long rows, int D) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (d < D)
    for (long long k = g; k < rows; k += 8) s += partial[k * D + d];
  part[g][lane] = s;
  __syncthreads();
  if (g > 0 || d >= D) return;
  for (int k = 1; k < 8; ++k) s += part[k][lane];
  // the ratio tends to one as both underflow
  const float sp = softplus(lam[d]);
  d_lam[d] = s * (sp > 0.f ? 1.0f / ((1.0f + expf(-lam[d])) * sp) : 1.f);
}

// ---- one token -------------------------------------------------------------

template <typename Ti, typename Th>
__global__ void __launch_bounds__(128)
glr_step_kernel(const Ti* __restrict__ x, const Ti* __restrict__ r, const Ti* __restrict__ i,
                const float* __restrict__ lam, float c, const float* state, float* state_out,
                Th* h, int D, int groups) {
  const int d = (blockIdx.x % groups) * 128 + threadIdx.x;
  if (d >= D) return;
  const size_t at = static_cast<size_t>(blockIdx.x / groups) * D + d;
  float a, root;
  decay(c * softplus(lam[d]) * sigmoid(Io<Ti>::ld(r, at)), a, root);
  const float v = root * sigmoid(Io<Ti>::ld(i, at)) * Io<Ti>::ld(x, at);
  const float st = fmaf(a, state[at], v);
  state_out[at] = st;
  if (h) Io<Th>::st(h, at, st);
}

// ---- launches --------------------------------------------------------------

template <typename F>
cudaError_t by_type(DType t, F&& f) {
  return t == DType::F32 ? f(float{}) : f(__nv_bfloat16{});
}
template <typename F>
cudaError_t by_mode(DType in_t, int D, F&& f) {
  const int e = in_t == DType::F32 ? 4 : 2;
  if (D * static_cast<long long>(e) % 16 == 0) return f(std::integral_constant<int, kWide>{});
  if (D % 2 == 0) return f(std::integral_constant<int, kEven>{});
  return f(std::integral_constant<int, kOdd>{});
}

// CTAs per cluster: the split of time that ends first when `resident` CTAs run
// at once, each round taking the same time.
int split_of(int nseq, long long Ttot, int D, int resident) {
#ifdef GLR_SPLIT
  return GLR_SPLIT;
#endif
  const long long pairs = static_cast<long long>((D + kChan - 1) / kChan) * nseq;
  const long long tiles = (Ttot + static_cast<long long>(nseq) * kTile - 1) / (static_cast<long long>(nseq) * kTile);
  int best = 1;
  long long cost = -1;
  for (int s = 1; s <= kMaxSplit && (s == 1 || s < 2 * tiles); s *= 2) {
    const long long waves = (pairs * s + resident - 1) / resident;
    const long long c = waves * ((tiles + s - 1) / s);
    if (cost < 0 || c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}
constexpr int kFwdResident = 3 * 148, kBwdResident = 1 * 148;

// Fills the common arguments and launches `kern` on clusters of `split` CTAs.
template <typename... P, typename... A>
cudaError_t launch_split(void (*kern)(P...), size_t smem, long long blocks, int split,
                         cudaStream_t s, A... args) {
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e == cudaSuccess && split > 8)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace

long long glr_bwd_partial_rows(int nseq, long long Ttot, int D) {
  return static_cast<long long>(nseq) * split_of(nseq, Ttot, D, kBwdResident);
}

cudaError_t launch_glr_fwd(const void* x, const void* r, const void* i, DType in_t,
                           const float* lam, float c, const SeqLayout& L, const float* state_in,
                           float* state_out, void* h, DType h_t, float* chunk_states, int D,
                           unsigned* err, cudaStream_t s) {
  Args p{x, r, i, lam, c, L, D, (D + kChan - 1) / kChan,
         split_of(L.nseq, L.Ttot, D, kFwdResident), err};
  const long long blocks = static_cast<long long>(p.groups) * L.nseq * p.split;
  return by_type(in_t, [&](auto ti) {
    return by_type(h_t, [&](auto th) {
      return by_mode(in_t, D, [&](auto mode) {
        using Ti = decltype(ti);
        using Th = decltype(th);
        constexpr int M = decltype(mode)::value;
        const size_t smem =
            warp_maps_bytes() + cta_maps_bytes(p.split) +
            (staged<Ti, M>() ? 2 * 3 * kTile * row_bytes<Ti>() : 0);
        return launch_split(glr_fwd_kernel<Ti, Th, M>, smem, blocks, p.split, s, p, state_in,
                            state_out, static_cast<Th*>(h), chunk_states);
      });
    });
  });
}

cudaError_t launch_glr_bwd(const void* x, const void* r, const void* i, DType in_t,
                           const float* lam, float c, const SeqLayout& L,
                           const float* chunk_states, const void* d_h, DType dh_t,
                           const float* d_state_out, void* dx, void* dr, void* di, DType g_t,
                           float* d_lam, float* d_state_in, float* partial, int D, unsigned* err,
                           cudaStream_t s) {
  Args p{x, r, i, lam, c, L, D, (D + kChan - 1) / kChan,
         split_of(L.nseq, L.Ttot, D, kBwdResident), err};
  const long long blocks = static_cast<long long>(p.groups) * L.nseq * p.split;
  const cudaError_t e = by_type(in_t, [&](auto ti) {
    return by_type(dh_t, [&](auto tu) {
      return by_type(g_t, [&](auto tg) {
        return by_mode(in_t, D, [&](auto mode) {
          using Ti = decltype(ti);
          using Tu = decltype(tu);
          using Tg = decltype(tg);
          constexpr int M = decltype(mode)::value;
          const size_t smem = warp_maps_bytes() + cta_maps_bytes(p.split) +
                              2 * kWarps * 32 * sizeof(float2) +
                              2 * kTile * (3 * row_bytes<Ti>() + row_bytes<Tu>());
          return launch_split(glr_bwd_kernel<Ti, Tu, Tg, M>, smem, blocks, p.split, s, p,
                              chunk_states, static_cast<const Tu*>(d_h), d_state_out,
                              static_cast<Tg*>(dx), static_cast<Tg*>(dr), static_cast<Tg*>(di),
                              d_state_in, partial);
        });
      });
    });
  });
  if (e != cudaSuccess) return e;
  glr_dlam_kernel<<<(D + 31) / 32, 256, 0, s>>>(partial, lam, d_lam,
                                                static_cast<long long>(L.nseq) * p.split, D);
  return cudaGetLastError();
}

cudaError_t launch_glr_step(const void* x, const void* r, const void* i, DType in_t,
                            const float* lam, float c, const float* state, float* state_out,
                            void* h, DType h_t, int N, int D, cudaStream_t s) {
  const int groups = (D + 127) / 128;
  const long long blocks = static_cast<long long>(groups) * N;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return by_type(in_t, [&](auto ti) {
    return by_type(h_t, [&](auto th) {
      using Ti = decltype(ti);
      using Th = decltype(th);
      glr_step_kernel<Ti, Th><<<static_cast<unsigned>(blocks), 128, 0, s>>>(
          static_cast<const Ti*>(x), static_cast<const Ti*>(r), static_cast<const Ti*>(i), lam, c,
          state, state_out, static_cast<Th*>(h), D, groups);
      return cudaGetLastError();
    });
  });
}

}  // namespace ret
