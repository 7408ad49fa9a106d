// Gated linear recurrence (ql.gl blog on Griffin/Hawk, section "Hawk"):
//     h_t = a_t h_(t-1) + b_t x_t, element by element, with
//     s = sigmoid(r), y = c softplus(lam) s, a = exp(-y), b = sqrt(1 - a^2) sigmoid(i),
// its gradients, and the one-token step.
//
// A token is the affine map h -> a h + v (v = b x), and a run of tokens is one
// too: (A, V) then (a, v) is (a A, a V + v).  So time is split: a CTA takes 64
// channels and 64 tokens per round, a warp 16 (gradients: 8) of those tokens, and
// a cluster of S CTAs 64 S consecutive tokens.  Every warp forms the map of its
// run from registers, the maps of the CTA's runs meet in shared memory and those
// of the cluster's CTAs are sent to each other's shared memory (st.async on an
// mbarrier); each warp then applies its tokens to the state that enters them.
// Every input is read from HBM once and every output written once.  The
// gradients run the same scheme from the last round to the first on
// e -> a (dh + e), with the forward's states formed again from the state that
// enters each 64-token tile, which the forward stored.  The inputs of the next
// round are copied to shared memory (cp.async) while the current one is computed.
//
// Measured at 2 x 8192 x 4096 bf16: forward 0.134 ms for 0.54 GB (61 % of the measured
// copy rate), gradients 0.266 ms for 0.94 GB (54 %).  Neither HBM nor a pipe is full
// (special functions 56 %, issue 50 %; gradients 36 % and 65 %): a round is a chain of ~2 us (gates,
// block barrier, exchange, apply), and with 128 registers and 256 CTAs an SM has fewer than two CTAs
// to overlap, unevenly (256 on 148).  With 16 sequences of 1024 tokens, the same bytes, no
// exchange and a full SM, the times are 0.101 ms (82 %) and 0.213 ms (68 %).  Deeper prefetch (3 or
// 4 stages), 32-channel CTAs, 8 warps of 8 tokens forward, results that leave through shared memory
// in 16-byte pieces and computing the next round's gates before the exchange is awaited
// changed the first case by less than 5 %, or made it slower.
#include <cmath>
#include <type_traits>

#include "launch.h"
#include "tc_ptx.cuh"

namespace ret {
namespace {

constexpr int kTile = kGlrChunk;    // tokens of a CTA per round
constexpr int kChan = 64;           // channels of a CTA: two per lane
constexpr int kMaxSplit = 16;       // CTAs of a cluster
// Warps of a CTA, and the consecutive tokens (run) of each.  Long runs share the cost of
// a round's exchange; the gradients keep three times as much per token in registers.
constexpr int kFwdWarps = 4, kFwdRun = kTile / kFwdWarps;
constexpr int kBwdWarps = 8, kBwdRun = kTile / kBwdWarps;
// Rounds whose rows are in shared memory at once.  Two of float32 would leave room for only one
// CTA of the gradients on an SM (0.213 ms instead of 0.185 ms at 2 x 8192 x 2048, 0.106 instead of
// 0.079 ms at 17 sequences, 9001 tokens x 1001).  The forward gains at these (0.089 instead of 0.093 and
// 0.049 instead of 0.051 ms) and loses where SMs are full (0.072 instead of 0.063 ms at 64 x 300 x
// 1001).  With one the next rows are on their way from the moment these have been read.
template <typename T> constexpr int stages() { return sizeof(T) == 2 ? 2 : 1; }

// How a lane's two channels lie and how rows reach shared memory.
//   kWide: channels 2l, 2l+1; rows start on 16-byte boundaries (D e bytes divide by 16)
//   kEven: channels 2l, 2l+1 (D even)
//   kOdd:  channels l, l+32
// All rows are copied in 16-byte pieces; those of kEven and kOdd may start inside their first one
// and have one piece more.
enum { kWide = 0, kEven = 1, kOdd = 2 };

// ---- pairs of floats (one instruction for both) ------------------------------

using F2 = float2;
__device__ __forceinline__ F2 f2(float x) { return make_float2(x, x); }
__device__ __forceinline__ F2 mul(F2 a, F2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ F2 add(F2 a, F2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) { return __ffma2_rn(a, b, c); }
// The same, or one instruction per channel: the gradients of float32 rows, and of bf16 rows whose
// channels come apart (kOdd), need fewer registers and are faster so, 0.185 ms instead of 0.192 ms
// at 2 x 8192 x 2048 float32.  Packed, bf16 takes 0.266 instead of 0.275 ms at 2 x 8192 x 4096, and
// the forward there 0.135 instead of 0.150 ms (float32 at 2 x 8192 x 2048 0.093 instead of 0.094).
template <bool PACKED> struct Pairs {
  static __device__ __forceinline__ F2 mul(F2 a, F2 b) {
    if constexpr (PACKED) return __fmul2_rn(a, b);
    return make_float2(a.x * b.x, a.y * b.y);
  }
  static __device__ __forceinline__ F2 add(F2 a, F2 b) {
    if constexpr (PACKED) return __fadd2_rn(a, b);
    return make_float2(a.x + b.x, a.y + b.y);
  }
  static __device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    if constexpr (PACKED) return __ffma2_rn(a, b, c);
    return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
  }
};

// ---- gates -----------------------------------------------------------------

__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// The gates are written for one channel: a packed operation takes four cycles of the FMA pipe
// for its two results (two single ones take two) and needs its constants in register pairs, while
// single ones take them as immediates.  Packed operations serve where only registers meet.
__device__ __forceinline__ float sigmoid(float x) {
  return rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * x));
}
__device__ __forceinline__ F2 sigmoid(F2 x) { return make_float2(sigmoid(x.x), sigmoid(x.y)); }

// c softplus(lam), at most the largest float: an infinite scale times the sigmoid of a closed gate
// (r = -inf, which also fills the last tile) or times a decay of zero would be NaN.  sigmoid never
// exceeds one, so y stays finite.
__device__ __forceinline__ float gate_scale(float c, float lam) {
  return min_nan(c * softplus(lam), 3.402823466e38f);
}
__device__ __forceinline__ F2 gate_scale(float c, F2 lam) {
  return make_float2(gate_scale(c, lam.x), gate_scale(c, lam.y));
}

// a = exp(-y) and root = sqrt(1 - a^2) for y >= 0, both to a few units of their
// own last place.  y = n ln 2 + g, |g| <= ln 2 / 2, and with w = 1 - e^-g = g + g^2 q(g)
// (q: the degree-4 polynomial of least largest error, found by reweighted least squares
// on Chebyshev points; w is off by a quarter of 2^-24) a = 2^-n - 2^-n w and
// 1 - a = 1 - 2^-n + 2^-n w, so 1 - a^2 = (1 - a)(1 + a) cancels nothing for decays
// near one.  From n = 127 on (y above 87.7, a below 8e-39) 2^-n is taken as zero,
// and root is zero where 1 - a^2 is below the normal range.
// SMALL: y is known to be at most kSmall, so n = 0: the same bits from half the work.  A CTA takes the
// general form where one of its channels needs it, and in the last group where D is no multiple of
// 64; all channels in it, 2 x 8192 x 4096 bf16 takes 155 / 284 us forward / gradients instead of
// 134 / 266, 16 x 1024 x 4096 109 / 228 instead of 101 / 213.
constexpr float kSmall = 0.3465f;
template <bool SMALL>
__device__ __forceinline__ void decay(float y, float& a, float& root) {
  float g = y, s = 1.f;
  if constexpr (!SMALL) {
    constexpr float kMagic = 12582912.f;           // 1.5 * 2^23: adding it rounds to an integer
    y = min_nan(y, 88.f);
    const float m = fmaf(y, -1.4426950408889634f, kMagic);     // kMagic - n
    const float n = m - kMagic;
    g = fmaf(n, 0.693147182464599609375f, y);                  // ln 2 in two parts
    g = fmaf(n, -1.904654290582768e-9f, g);
    s = __int_as_float((__float_as_int(m) << 23) + 0x3f800000);
  }
  float w = fmaf(g, -0.0013945651007816195f, 0.008366155438125134f);
  w = fmaf(g, w, -0.04166629537940025f);
  w = fmaf(g, w, 0.1666654795408249f);
  w = fmaf(g, w, -0.5f);
  w = fmaf(g * g, w, g);
  float below = w;                                 // 1 - a
  if constexpr (SMALL) {
    a = 1.f - w;
  } else {
    a = fmaf(-s, w, s);
    below = fmaf(s, w, 1.f - s);
  }
  root = sqrt_approx(fmaf(below, a, below));
}
template <bool SMALL>
__device__ __forceinline__ void decay(F2 y, F2& a, F2& root) {
  decay<SMALL>(y.x, a.x, root.x);
  decay<SMALL>(y.y, a.y, root.y);
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

// Copies `bytes` and fills the rest of the 16 with zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Bytes of a staged row, and of a warp's rows of one array.
template <typename T, int MODE> constexpr int row_bytes() {
  return kChan * static_cast<int>(sizeof(T)) + (MODE == kWide ? 0 : 16);
}
template <typename T, int MODE, int RUN> constexpr int run_bytes() {
  return RUN * row_bytes<T, MODE>();
}
// Elements by which row t lies inside its first piece (c0 is a multiple of a piece).
template <typename T, int MODE> __device__ __forceinline__ int row_shift(int t, int D) {
  if constexpr (MODE == kWide) return 0;
  return static_cast<int>(static_cast<unsigned>(t) * static_cast<unsigned>(D) &
                          (16 / sizeof(T) - 1));
}

// Copies a warp's rows t .. t+RUN-1, channels c0 .. c0+63, of N arrays of one shape to `dst`, one
// run_bytes after the other; rows at or past t1 are filled with `fill` (two bf16, or the float)
// instead: r = -inf, and zeros elsewhere, make a token the identity.  `total` is the tensor's
// element count: nothing past it is read.  (4-byte pieces, which fit every row, took 0.147 ms
// instead of 0.052 ms forward and 0.182 instead of 0.098 ms for the gradients at 8192 x 1001 bf16.)
template <typename T, int MODE, int RUN, int N>
__device__ __forceinline__ void stage_rows(char* dst, const T* const (&src)[N],
                                           const uint32_t (&fill)[N], int t, int t1, int c0, int D,
                                           size_t total, int lane) {
  constexpr int kElems = 16 / static_cast<int>(sizeof(T));
  constexpr int kPer = kChan / kElems;                    // pieces of a row, without the last
  constexpr int kStep = 32 / kPer;                        // rows per access of the warp
  constexpr int kArray = run_bytes<T, MODE, RUN>();
  const int width = min(kChan, D - c0);
  const auto piece = [&](int row, int q) {
    char* to = dst + row * row_bytes<T, MODE>() + q * 16;
    if (t + row >= t1) {
#pragma unroll
      for (int n = 0; n < N; ++n)
        *reinterpret_cast<uint4*>(to + n * kArray) =
            make_uint4(fill[n], fill[n], fill[n], fill[n]);
      return;
    }
    const size_t at = static_cast<size_t>(t + row) * D + c0;
    const int in = q * kElems - row_shift<T, MODE>(t + row, D);      // first channel of the piece
    if (in >= width) return;
    const size_t from = at + in;
    const int bytes =
        MODE == kWide ? 16
                      : static_cast<int>(min(static_cast<size_t>(kElems), total - from)) *
                            static_cast<int>(sizeof(T));
#pragma unroll
    for (int n = 0; n < N; ++n)
      cp_async16(tc::smem_u32(to + n * kArray), src[n] + from, bytes);
  };
#pragma unroll
  for (int k = 0; k < RUN / kStep; ++k) piece(k * kStep + lane / kPer, lane % kPer);
  if constexpr (MODE != kWide) {
    static_assert(RUN <= 32, "one last piece per lane");
    if (lane < RUN) piece(lane, kPer);
  }
}

// kWide, a run that lies whole inside the sequence: `from` is the lane's first piece
// (stage_from), the copies differ by whole rows only.
template <typename T>
__device__ __forceinline__ const T* stage_from(const T* src, int t, int c0, int D, int lane) {
  constexpr int kElems = 16 / static_cast<int>(sizeof(T)), kPer = kChan / kElems;
  return src + static_cast<ptrdiff_t>(t + lane / kPer) * D + c0 + lane % kPer * kElems;
}
template <typename T, int RUN>
__device__ __forceinline__ void stage_full(char* dst, const T* from, int c0, int D, int lane) {
  constexpr int kElems = 16 / static_cast<int>(sizeof(T)), kPer = kChan / kElems;
  constexpr int kStep = 32 / kPer;
  if (c0 + lane % kPer * kElems >= D) return;
  const uint32_t d = tc::smem_u32(dst) + lane * 16;
#pragma unroll
  for (int k = 0; k < RUN / kStep; ++k)
    cp_async16(d + k * 512, from + static_cast<ptrdiff_t>(k * kStep) * D, 16);
}

// A lane's two channels of staged row k, token t.
template <typename T, int MODE>
__device__ __forceinline__ F2 row_pair(const char* st, int k, int t, int D, int lane) {
  const char* row = st + k * row_bytes<T, MODE>() +
                    row_shift<T, MODE>(t, D) * static_cast<int>(sizeof(T));
  if constexpr (MODE == kOdd && sizeof(T) == 2) {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(row);
    return make_float2(__uint_as_float(static_cast<uint32_t>(q[lane]) << 16),
                       __uint_as_float(static_cast<uint32_t>(q[lane + 32]) << 16));
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(row + lane * 4);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  } else if constexpr (MODE == kOdd) {
    const float* q = reinterpret_cast<const float*>(row);
    return make_float2(q[lane], q[lane + 32]);
  } else {
    return *reinterpret_cast<const F2*>(row + lane * 8);
  }
}

// Two floats per lane in the place of row k of the r array (and, for bf16, of the i array, which
// follows at `array` bytes).
template <typename T, int MODE>
__device__ __forceinline__ void put_state(char* st, int array, int k, int lane, F2 v) {
  char* row = st + array + k * row_bytes<T, MODE>();
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<float*>(row + lane * 4) = v.x;
    *reinterpret_cast<float*>(row + array + lane * 4) = v.y;
  } else {
    *reinterpret_cast<F2*>(row + lane * 8) = v;
  }
}
template <typename T, int MODE>
__device__ __forceinline__ F2 get_state(const char* st, int array, int k, int lane) {
  const char* row = st + array + k * row_bytes<T, MODE>();
  if constexpr (sizeof(T) == 2)
    return make_float2(*reinterpret_cast<const float*>(row + lane * 4),
                       *reinterpret_cast<const float*>(row + array + lane * 4));
  else
    return *reinterpret_cast<const F2*>(row + lane * 8);
}

// `at`: offset of the lane's first channel.
template <typename T, int MODE>
__device__ __forceinline__ void store_pair(T* at, F2 v, bool okA, bool okB) {
  if constexpr (MODE == kOdd) {
    if (okA) Io<T>::st(at, 0, v.x);
    if (okB) Io<T>::st(at, 32, v.y);
  } else if (okA) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<__nv_bfloat162*>(at) = __floats2bfloat162_rn(v.x, v.y);
    else
      *reinterpret_cast<F2*>(at) = v;
  }
}

__device__ __forceinline__ F2 load2(const float* p, size_t at, int cA, int cB, int D) {
  return make_float2(p && cA < D ? p[at + cA] : 0.f, p && cB < D ? p[at + cB] : 0.f);
}
__device__ __forceinline__ void store2(float* p, size_t at, F2 v, int cA, int cB, int D) {
  if (cA < D) p[at + cA] = v.x;
  if (cB < D) p[at + cB] = v.y;
}

// ---- affine maps and their exchange -------------------------------------------

// h -> A h + V for a lane's two channels.
struct Map {
  F2 A, V;
};
__device__ __forceinline__ F2 apply(const Map& m, F2 h) { return fma(m.A, h, m.V); }
__device__ __forceinline__ Map then(const Map& m, const Map& n) {      // first m, then n
  return Map{mul(n.A, m.A), fma(n.A, m.V, n.V)};
}
__device__ __forceinline__ Map identity() { return Map{f2(1.f), f2(0.f)}; }

using Maps = float4[32];             // one map per lane
__device__ __forceinline__ Map get(const Maps& m, int lane) {
  const float4 v = m[lane];
  return Map{make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ float4 pack(const Map& m) {
  return make_float4(m.A.x, m.A.y, m.V.x, m.V.y);
}

// Shared memory of the exchange: per round parity, the maps of the CTA's warps
// and those of the cluster's CTAs, with a barrier that counts the latter's
// bytes.  A buffer is written again two rounds later; by then every reader has
// passed the block barrier (warp maps) of the round between, and a CTA sends its
// next map only after that, so a map received tells that the sender's warps have
// read everything of the round before last.  The maps and rows behind it start on 128-byte lines
// (16 bytes off 32, the forward of 2 x 8192 x 4096 took 0.152 ms instead of 0.135 ms).
struct alignas(128) Exchange {
  uint64_t bar[2];
  int abort;                            // a wait of this CTA has given up
  int seq;                              // of longest_first
  int sent;                             // rounds whose map this CTA has sent
  int failed;                           // a wait of any CTA has given up (set by it at the end)
  int all_sent[kMaxSplit];              // `sent` of every CTA, where one has failed
  int stop;                             // `abort` as the sending warp saw it before the round's barrier
};
__host__ __device__ constexpr size_t exchange_bytes(int split, int warps) {
  return sizeof(Exchange) + 2 * (warps + (split > 1 ? split : 0)) * sizeof(Maps);
}

__device__ __forceinline__ void st_async_f32x4(uint32_t remote, float4 v, uint32_t remote_bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 "
      "[%0], {%1, %2, %3, %4}, [%5];" ::"r"(remote),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(remote_bar)
      : "memory");
}

// The sequence of a cluster that is the slot-th to start: packed sequences go by length, the longest
// first (it ends last), where there are at most 128 of them; among more, one weighs less.  Every
// cluster ranks them for itself.  Forward / gradients in us in this order and in the given one: 17
// sequences of 9001 tokens x 1001 float32 51 / 79 and 58 / 108, 64 of 200000 x 1024 bf16 351 / 688 and
// 459 / 889.
constexpr int kMaxRanked = 128;
static_assert(kMaxRanked <= kFwdWarps * 32 && kMaxRanked <= kBwdWarps * 32, "a thread each");
__device__ __forceinline__ int longest_first(const SeqLayout& L, int slot, Exchange& ex,
                                             int* lengths) {
  if (L.cu == nullptr || L.nseq == 1 || L.nseq > kMaxRanked) return slot;
  const int s = threadIdx.x;
  int mine = 0;
  if (s == 0) ex.seq = slot;
  if (s < L.nseq) {
    int a, b;
    seq_bounds(L, s, a, b);
    lengths[s] = mine = b - a;
  }
  __syncthreads();
  if (s < L.nseq) {
    int before = 0;
#pragma unroll 4
    for (int q = 0; q < L.nseq; ++q) {
      const int other = lengths[q];
      before += other > mine || (other == mine && q < s);
    }
    if (before == slot) ex.seq = s;
  }
  __syncthreads();
  return ex.seq;
}

// Start of a kernel, before anything is on its way: the fence makes these writes come before
// those that other CTAs make later.
__device__ __forceinline__ void exchange_init(Exchange& ex, int S) {
  if (S == 1 || threadIdx.x != 0) return;
  tc::mbar_init(&ex.bar[0], 1);
  tc::mbar_init(&ex.bar[1], 1);
  ex.abort = ex.sent = ex.failed = 0;
  tc::fence_barrier_init();
  tc::fence_cluster();
}
// Before the first map is sent: every CTA of the cluster is running and its barriers are set up.
__device__ __forceinline__ void exchange_begin(int S) {
  if (S == 1) return;
  __syncthreads();
  tc::cluster_arrive_relaxed();
  tc::cluster_wait();
}
__device__ __forceinline__ bool gave_up(const Exchange& ex) {
  return *static_cast<const volatile int*>(&ex.abort) != 0;
}
__device__ __forceinline__ void send_map(Exchange& ex, Maps* cta, const Map& mine, int n, int S,
                                         int rank, int lane) {
  Maps* to = cta + (n & 1) * S;
  uint64_t* bar = &ex.bar[n & 1];
  if (lane == 0) tc::mbar_arrive_expect_tx(bar, S * sizeof(Maps));
  for (int q = 0; q < S; ++q)
    st_async_f32x4(tc::cluster_addr(&to[rank][lane], q), pack(mine), tc::cluster_addr(bar, q));
}
// Before the block barrier of a round, by the warp that will send: all its lanes then read the same
// (a vote in `send` cost the gradients 64 bytes of spills).
__device__ __forceinline__ void send_or_stop(Exchange& ex, int S, int lane) {
  if (S > 1 && lane == 0) ex.stop = gave_up(ex);
}
// One warp sends its CTA's map of round `n` to every CTA of the cluster, unless a wait of this
// CTA has given up: so it has received every map of round n - 1, and no CTA is ever more than one
// round ahead of another.  The stores carry their own completion, so nothing here waits for
// stores to global memory (the release of a cluster barrier would: 0.38 ms instead of 0.27 ms at
// 2 x 8192 x 4096, forward).
__device__ __forceinline__ void send(Exchange& ex, Maps* cta, const Map& mine, int n, int S,
                                     int rank, int lane) {
  if (*static_cast<const volatile int*>(&ex.stop)) return;
  if (lane == 0) ex.sent = n + 1;
  send_map(ex, cta, mine, n, S, rank, lane);
}
// Waits for the maps of round `n`.  The wait is bounded; once one has run out the others
// return at once, the rounds go on without exchange and the error is reported.
__device__ __forceinline__ void receive(Exchange& ex, int n, unsigned* err) {
  if (gave_up(ex)) return;
  tc::mbar_wait_cluster(&ex.bar[n & 1], (n >> 1) & 1, &ex.abort, err);
}
// End of a kernel: no CTA leaves while maps may still be on their way to it.  Where no wait has
// given up, each CTA has received every map of every round.  Otherwise a CTA that gave up tells
// all of them; all tell each other how many rounds they have sent, those that are behind by the one
// round send it as well (its contents count for nothing), and each waits, bounded again, for
// the last two rounds, before which everything has arrived.
__device__ __forceinline__ void exchange_end(Exchange& ex, Maps* cta, int S, int rank) {
  if (S == 1) return;
  const int t = threadIdx.x;
  __syncthreads();                        // abort and sent are final
  if (t < S && ex.abort) {
    tc::st_cluster_s32(tc::cluster_addr(&ex.failed, t), 1);
    tc::fence_cluster();
  }
  tc::cluster_arrive_relaxed();
  tc::cluster_wait();
  if (!*static_cast<volatile int*>(&ex.failed)) return;
  if (t < S) {
    tc::st_cluster_s32(tc::cluster_addr(&ex.all_sent[rank], t), ex.sent);
    tc::fence_cluster();
  }
  tc::cluster_arrive_relaxed();
  tc::cluster_wait();
  const volatile int* all = ex.all_sent;
  int most = 0;
  for (int q = 0; q < S; ++q) most = max(most, all[q]);
  if (t < 32 && all[rank] < most) send_map(ex, cta, identity(), most - 1, S, rank, t);
  for (int n = max(most - 2, 0); n < most; ++n)
    tc::mbar_wait_drain(&ex.bar[n & 1], (n >> 1) & 1);
}

// ---- forward ---------------------------------------------------------------

template <typename Ti, typename Th, int MODE>
__global__ void __launch_bounds__(kFwdWarps * 32, 4)
glr_fwd_kernel(Args p, const float* __restrict__ state_in, float* __restrict__ state_out,
               Th* __restrict__ h, float* __restrict__ chunk_states) {
  extern __shared__ __align__(128) char smem[];
  constexpr int kWarps = kFwdWarps, kRun = kFwdRun;
  constexpr int kArray = run_bytes<Ti, MODE, kRun>(), kStages = stages<Ti>();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = p.split, rank = static_cast<int>(blockIdx.x % S);
  Exchange& ex = *reinterpret_cast<Exchange*>(smem);
  exchange_init(ex, S);
  Maps(*warp_maps)[kWarps] = reinterpret_cast<Maps(*)[kWarps]>(smem + sizeof(Exchange));   // [2]
  Maps* cta_maps = reinterpret_cast<Maps*>(warp_maps + 2);                // [2][S]
  char* ring = smem + exchange_bytes(S, kWarps) + warp * (kStages * 3 * kArray);
  const int pair = static_cast<int>(blockIdx.x / S);
  const int seq = longest_first(p.L, pair / p.groups, ex, reinterpret_cast<int*>(warp_maps));
  const int c0 = pair % p.groups * kChan;
  const int D = p.D;
  const int cA = c0 + (MODE == kOdd ? lane : 2 * lane), cB = MODE == kOdd ? cA + 32 : cA + 1;
  const bool okA = cA < D, okB = cB < D;
  const Ti* x = static_cast<const Ti*>(p.x);
  const Ti* r = static_cast<const Ti*>(p.r);
  const Ti* i = static_cast<const Ti*>(p.i);
  const size_t total = static_cast<size_t>(p.L.Ttot) * D;
  int t0, t1;
  seq_bounds(p.L, seq, t0, t1);
  if (c0 == 0 && rank == 0 && threadIdx.x == 0) check_offsets(p.L, seq, p.err);
  const int rounds = ceil_div(t1 - t0, kTile * S);
  const uint32_t minus_inf = sizeof(Ti) == 2 ? 0xff80ff80u : 0xff800000u;
  const auto first = [&](int j) { return t0 + ((j * S + rank) * kWarps + warp) * kRun; };
  const ptrdiff_t stride = static_cast<ptrdiff_t>(S) * kTile * D;          // of a round
  const Ti* const src[3] = {x, r, i};
  const uint32_t pad[3] = {0u, minus_inf, 0u};
  const Ti* from[3];                    // of the next fetch
#pragma unroll
  for (int n = 0; n < 3; ++n) from[n] = stage_from(src[n], first(0), c0, D, lane);
  const auto fetch = [&](int j) {
    if (j < rounds) {
      char* st = ring + j % kStages * 3 * kArray;
      const int t = first(j);
      if (MODE == kWide && t + kRun <= t1) {
#pragma unroll
        for (int n = 0; n < 3; ++n) stage_full<Ti, kRun>(st + n * kArray, from[n], c0, D, lane);
      } else {
        stage_rows<Ti, MODE, kRun>(st, src, pad, t, t1, c0, D, total, lane);
      }
#pragma unroll
      for (int n = 0; n < 3; ++n) from[n] += stride;
    }
    cp_commit();
  };
  fetch(0);
  const F2 lm = load2(p.lam, 0, cA, cB, D);
  const F2 ysc = gate_scale(p.c, lm);
  F2 carry = load2(state_in, static_cast<size_t>(seq) * D, cA, cB, D);
  exchange_begin(S);
  const auto run = [&](auto small) {
    for (int j = 0; j < rounds; ++j) {
      if (kStages > 1) fetch(j + 1);
      cp_wait<kStages - 1>();
      __syncwarp();
      const char* st = ring + j % kStages * 3 * kArray;
      const int t = first(j);
      F2 a[kRun], v[kRun];
      Map m = identity();
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const F2 xv = row_pair<Ti, MODE>(st, k, t + k, D, lane);
        const F2 rv = row_pair<Ti, MODE>(st + kArray, k, t + k, D, lane);
        const F2 iv = row_pair<Ti, MODE>(st + 2 * kArray, k, t + k, D, lane);
        F2 root;
        decay<decltype(small)::value>(mul(ysc, sigmoid(rv)), a[k], root);
        v[k] = mul(mul(root, sigmoid(iv)), xv);
        m = k == 0 ? Map{a[0], v[0]} : then(m, Map{a[k], v[k]});
      }
      __syncwarp();                       // the buffer refilled next was read to here
      if (kStages == 1) fetch(j + 1);
      Maps* wm = warp_maps[j & 1];
      wm[warp][lane] = pack(m);
      if (warp == kWarps - 1) send_or_stop(ex, S, lane);
      __syncthreads();
      F2 enter, hs;                       // the states that enter the tile and the warp's run
      if (S == 1) {
        enter = hs = carry;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w == warp) hs = carry;
          carry = apply(get(wm[w], lane), carry);
        }
      } else {
        Map before = identity();
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
          if (w < warp) before = then(before, get(wm[w], lane));
        if (warp == kWarps - 1) send(ex, cta_maps, then(before, m), j, S, rank, lane);
        receive(ex, j, p.err);
        const Maps* cm = cta_maps + (j & 1) * S;
        int q = 0;
#pragma unroll 4
        for (; q < rank; ++q) carry = apply(get(cm[q], lane), carry);
        enter = carry;
#pragma unroll 4
        for (; q < S; ++q) carry = apply(get(cm[q], lane), carry);
        hs = apply(before, enter);
      }
      if (chunk_states && warp == 0 && t < t1)
        store2(chunk_states, static_cast<size_t>(chunk_row(t0, seq) + j * S + rank) * D, enter, cA,
               cB, D);
      Th* out = h + static_cast<size_t>(t) * D + cA;
      if (t + kRun <= t1) {
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          hs = fma(a[k], hs, v[k]);
          store_pair<Th, MODE>(out + static_cast<ptrdiff_t>(k) * D, hs, okA, okB);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          hs = fma(a[k], hs, v[k]);
          if (t + k < t1) store_pair<Th, MODE>(out + static_cast<ptrdiff_t>(k) * D, hs, okA, okB);
        }
      }
    }
  };
  // every warp of the CTA has the same 64 channels, so all take the same way
  if (__all_sync(0xffffffffu, ysc.x <= kSmall && ysc.y <= kSmall))
    run(std::true_type{});
  else
    run(std::false_type{});
  if (state_out && rank == 0 && warp == 0)
    store2(state_out, static_cast<size_t>(seq) * D, carry, cA, cB, D);
  exchange_end(ex, cta_maps, S, rank);
}

// ---- gradients -------------------------------------------------------------

// A token's gradients from G = d_h + e, the e it passes on (a G) and the state before it.
template <typename P>
__device__ __forceinline__ void gate_gradients(F2 G, F2 e, F2 a, F2 root, F2 y, F2 sr, F2 si, F2 x,
                                               F2 hp, F2& gx, F2& gr, F2& gi, F2& u) {
  // 1 / root; where root is zero y is below 1e-38 and y / root counts as zero either way
  const F2 inv = make_float2(rcp_approx(fmaxf(root.x, 1e-19f)), rcp_approx(fmaxf(root.y, 1e-19f)));
  const F2 six = P::mul(si, x), ai = P::mul(a, inv);
  gx = P::mul(G, P::mul(root, si));
  const F2 gix = P::mul(gx, x);
  gi = make_float2(fmaf(gix.x, -si.x, gix.x), fmaf(gix.y, -si.y, gix.y));
  u = P::mul(P::mul(e, y), make_float2(fmaf(ai.x, six.x, -hp.x), fmaf(ai.y, six.y, -hp.y)));
  gr = make_float2(fmaf(u.x, -sr.x, u.x), fmaf(u.y, -sr.y, u.y));
}

template <typename Ti, typename Tu, typename Tg, int MODE>
__global__ void __launch_bounds__(kBwdWarps * 32, 2)
glr_bwd_kernel(Args p, const float* __restrict__ chunk_states, const Tu* __restrict__ dh,
               const float* __restrict__ d_state_out, Tg* __restrict__ dx, Tg* __restrict__ dr,
               Tg* __restrict__ di, float* __restrict__ d_state_in, float* __restrict__ partial) {
  extern __shared__ __align__(128) char smem[];
  using P = Pairs<sizeof(Ti) == 2 && MODE != kOdd>;
  constexpr int kWarps = kBwdWarps, kRun = kBwdRun;
  constexpr int kArray = run_bytes<Ti, MODE, kRun>(), kUp = run_bytes<Tu, MODE, kRun>();
  constexpr int kStage = 3 * kArray + kUp, kStages = stages<Ti>();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = p.split, rank = static_cast<int>(blockIdx.x % S);
  Exchange& ex = *reinterpret_cast<Exchange*>(smem);
  exchange_init(ex, S);
  Maps(*warp_maps)[kWarps] = reinterpret_cast<Maps(*)[kWarps]>(smem + sizeof(Exchange));   // [2]
  Maps* cta_maps = reinterpret_cast<Maps*>(warp_maps + 2);                // [2][S]
  F2(*wf)[kWarps][32] = reinterpret_cast<F2(*)[kWarps][32]>(smem + exchange_bytes(S, kWarps));
  char* ring = reinterpret_cast<char*>(wf + 2) + warp * (kStages * kStage);
  const int pair = static_cast<int>(blockIdx.x / S);
  const int seq = longest_first(p.L, pair / p.groups, ex, reinterpret_cast<int*>(warp_maps));
  const int c0 = pair % p.groups * kChan;
  const int D = p.D;
  const int cA = c0 + (MODE == kOdd ? lane : 2 * lane), cB = MODE == kOdd ? cA + 32 : cA + 1;
  const bool okA = cA < D, okB = cB < D;
  const Ti* x = static_cast<const Ti*>(p.x);
  const Ti* r = static_cast<const Ti*>(p.r);
  const Ti* i = static_cast<const Ti*>(p.i);
  const size_t total = static_cast<size_t>(p.L.Ttot) * D;
  int t0, t1;
  seq_bounds(p.L, seq, t0, t1);
  if (c0 == 0 && rank == 0 && threadIdx.x == 0) check_offsets(p.L, seq, p.err);
  const int rounds = ceil_div(t1 - t0, kTile * S);
  const uint32_t minus_inf = sizeof(Ti) == 2 ? 0xff80ff80u : 0xff800000u;
  const auto first = [&](int j) { return t0 + ((j * S + rank) * kWarps + warp) * kRun; };
  const Ti* const src[3] = {x, r, i};
  const uint32_t pad[3] = {0u, minus_inf, 0u};
  const Tu* const src_u[1] = {dh};
  const uint32_t pad_u[1] = {0u};
  const auto fetch = [&](int j) {
    if (j >= 0) {
      char* st = ring + j % kStages * kStage;
      stage_rows<Ti, MODE, kRun>(st, src, pad, first(j), t1, c0, D, total, lane);
      stage_rows<Tu, MODE, kRun>(st + 3 * kArray, src_u, pad_u, first(j), t1, c0, D, total, lane);
    }
    cp_commit();
  };
  const auto entering = [&](int j) {
    const int tile = j * S + rank;
    if (j < 0 || t0 + tile * kTile >= t1) return f2(0.f);
    return load2(chunk_states, static_cast<size_t>(chunk_row(t0, seq) + tile) * D, cA, cB, D);
  };
  fetch(rounds - 1);
  F2 cs = entering(rounds - 1);
  const F2 lm = load2(p.lam, 0, cA, cB, D);
  const F2 ysc = gate_scale(p.c, lm);
  const size_t so = static_cast<size_t>(seq) * D;
  F2 carry = load2(d_state_out, so, cA, cB, D);
  F2 usum = f2(0.f);
  exchange_begin(S);
  const auto run = [&](auto small) {
    for (int j = rounds - 1; j >= 0; --j) {
      const int n = rounds - 1 - j;
      if (kStages > 1) fetch(j - 1);
      const F2 cs_next = entering(j - 1);
      cp_wait<kStages - 1>();
      __syncwarp();
      const char* st = ring + j % kStages * kStage;
      const int t = first(j);
      // the run's map of h forwards (fw) and of e backwards (the same product, sum w)
      F2 a[kRun], root[kRun], sr[kRun], si[kRun];
      Map fw = identity();
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const F2 xv = row_pair<Ti, MODE>(st, k, t + k, D, lane);
        const F2 rv = row_pair<Ti, MODE>(st + kArray, k, t + k, D, lane);
        const F2 iv = row_pair<Ti, MODE>(st + 2 * kArray, k, t + k, D, lane);
        sr[k] = sigmoid(rv);
        si[k] = sigmoid(iv);
        decay<decltype(small)::value>(P::mul(ysc, sr[k]), a[k], root[k]);
        const Map m = Map{a[k], P::mul(P::mul(root[k], si[k]), xv)};
        fw = k == 0 ? m : then(fw, m);
      }
      F2 w = f2(0.f);
#pragma unroll
      for (int k = kRun - 1; k >= 0; --k)
        w = P::mul(a[k], P::add(row_pair<Tu, MODE>(st + 3 * kArray, k, t + k, D, lane), w));
      Maps* wm = warp_maps[n & 1];
      wm[warp][lane] = pack(Map{fw.A, w});
      wf[n & 1][warp][lane] = fw.V;
      if (warp == 0) send_or_stop(ex, S, lane);
      __syncthreads();
      F2 hs = cs, e;                      // the state and the gradient that enter the run
#pragma unroll 1
      for (int q = 0; q < warp; ++q) hs = P::fma(get(wm[q], lane).A, hs, wf[n & 1][q][lane]);
      if (S == 1) {
        e = carry;
#pragma unroll
        for (int q = kWarps - 1; q >= 0; --q) {
          if (q == warp) e = carry;
          carry = apply(get(wm[q], lane), carry);
        }
      } else {
        Map after = identity();
#pragma unroll 1
        for (int q = kWarps - 1; q > warp; --q) after = then(after, get(wm[q], lane));
        if (warp == 0) send(ex, cta_maps, then(after, Map{fw.A, w}), n, S, rank, lane);
        receive(ex, n, p.err);
        const Maps* cm = cta_maps + (n & 1) * S;
        int q = S - 1;
#pragma unroll 4
        for (; q > rank; --q) carry = apply(get(cm[q], lane), carry);
        e = apply(after, carry);
#pragma unroll 4
        for (; q >= 0; --q) carry = apply(get(cm[q], lane), carry);
      }
      // the state before each token, kept where the token's gate inputs were (every lane has read
      // its own; odd rows share pieces, but all lanes are past the block barrier)
      char* keep = ring + j % kStages * kStage;
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        put_state<Ti, MODE>(keep, kArray, k, lane, hs);
        const F2 xv = row_pair<Ti, MODE>(st, k, t + k, D, lane);
        if (k + 1 < kRun) hs = P::fma(a[k], hs, P::mul(P::mul(root[k], si[k]), xv));
      }
      const size_t at = static_cast<size_t>(t) * D + cA;
#pragma unroll
      for (int k = kRun - 1; k >= 0; --k) {
        const F2 xv = row_pair<Ti, MODE>(st, k, t + k, D, lane);
        const F2 hp = get_state<Ti, MODE>(keep, kArray, k, lane);
        const F2 G = P::add(row_pair<Tu, MODE>(st + 3 * kArray, k, t + k, D, lane), e);
        F2 gx, gr, gi, u;
        e = P::mul(a[k], G);
        gate_gradients<P>(G, e, a[k], root[k], P::mul(ysc, sr[k]), sr[k], si[k], xv, hp, gx, gr, gi,
                          u);
        usum = P::add(usum, u);
        if (t + k < t1) {
          const size_t o = at + static_cast<size_t>(k) * D;
          store_pair<Tg, MODE>(dx + o, gx, okA, okB);
          store_pair<Tg, MODE>(dr + o, gr, okA, okB);
          store_pair<Tg, MODE>(di + o, gi, okA, okB);
        }
      }
      cs = cs_next;
      __syncwarp();                       // the buffer refilled next was read to here
      if (kStages == 1) fetch(j - 1);
    }
  };
  // every warp of the CTA has the same 64 channels, so all take the same way
  if (__all_sync(0xffffffffu, ysc.x <= kSmall && ysc.y <= kSmall))
    run(std::true_type{});
  else
    run(std::false_type{});
  if (d_state_in && rank == 0 && warp == 0) store2(d_state_in, so, carry, cA, cB, D);
  // this CTA's part of sum u, its warps in order
  __syncthreads();
  wf[0][warp][lane] = usum;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int q = 1; q < kWarps; ++q) usum = P::add(usum, wf[0][q][lane]);
    store2(partial, (static_cast<size_t>(seq) * S + rank) * D, usum, cA, cB, D);
  }
  exchange_end(ex, cta_maps, S, rank);
}

// ---- short sequences ------------------------------------------------------------
//
// A thread takes two channels of one sequence through time, and nothing is exchanged.  Eight tokens
// are loaded at a time.

constexpr int kDirectThreads = 128, kDirectChan = 2 * kDirectThreads, kBatch = 8;

// Two channels of a row: adjacent (PAIR), or kDirectThreads apart.
template <typename T, bool PAIR>
__device__ __forceinline__ F2 load_two(const T* row, bool okA, bool okB) {
  if constexpr (PAIR) {
    if (!okA) return f2(0.f);
    if constexpr (sizeof(T) == 2) {
      const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(row));
      return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
      return __ldg(reinterpret_cast<const F2*>(row));
    }
  } else {
    return make_float2(okA ? Io<T>::ld(row, 0) : 0.f, okB ? Io<T>::ld(row, kDirectThreads) : 0.f);
  }
}
template <typename T, bool PAIR>
__device__ __forceinline__ void store_two(T* row, F2 v, bool okA, bool okB) {
  if constexpr (PAIR) {
    if (!okA) return;
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<__nv_bfloat162*>(row) = __floats2bfloat162_rn(v.x, v.y);
    else
      *reinterpret_cast<F2*>(row) = v;
  } else {
    if (okA) Io<T>::st(row, 0, v.x);
    if (okB) Io<T>::st(row, kDirectThreads, v.y);
  }
}

template <typename Ti, typename Th, bool PAIR>
__global__ void __launch_bounds__(kDirectThreads)
glr_fwd_direct_kernel(Args p, const float* __restrict__ state_in, float* __restrict__ state_out,
                      Th* __restrict__ h, float* __restrict__ chunk_states) {
  const int D = p.D;
  const int seq = static_cast<int>(blockIdx.x / p.groups);
  const int c0 = static_cast<int>(blockIdx.x % p.groups) * kDirectChan;
  const int cA = c0 + (PAIR ? 2 : 1) * static_cast<int>(threadIdx.x);
  const int cB = cA + (PAIR ? 1 : kDirectThreads);
  const bool okA = cA < D, okB = cB < D;
  if (c0 == 0 && threadIdx.x == 0) check_offsets(p.L, seq, p.err);
  if (!okA) return;
  int t0, t1;
  seq_bounds(p.L, seq, t0, t1);
  const F2 lm = load2(p.lam, 0, cA, cB, D);
  const F2 ysc = gate_scale(p.c, lm);
  F2 st = load2(state_in, static_cast<size_t>(seq) * D, cA, cB, D);
  size_t at = static_cast<size_t>(t0) * D + cA;
  for (int t = t0; t < t1; t += kBatch) {
    F2 x[kBatch], r[kBatch], i[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const bool in = t + k < t1;
      const size_t o = at + static_cast<size_t>(k) * D;
      x[k] = load_two<Ti, PAIR>(static_cast<const Ti*>(p.x) + o, in, in && okB);
      r[k] = load_two<Ti, PAIR>(static_cast<const Ti*>(p.r) + o, in, in && okB);
      i[k] = load_two<Ti, PAIR>(static_cast<const Ti*>(p.i) + o, in, in && okB);
    }
    if (chunk_states && (t - t0) % kGlrChunk == 0)
      store2(chunk_states, static_cast<size_t>(chunk_row(t0, seq) + (t - t0) / kGlrChunk) * D, st, cA,
             cB, D);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (t + k >= t1) break;
      F2 a, root;
      decay<false>(mul(ysc, sigmoid(r[k])), a, root);
      st = fma(a, st, mul(mul(root, sigmoid(i[k])), x[k]));
      store_two<Th, PAIR>(h + at + static_cast<size_t>(k) * D, st, true, okB);
    }
    at += static_cast<size_t>(kBatch) * D;
  }
  if (state_out) store2(state_out, static_cast<size_t>(seq) * D, st, cA, cB, D);
}

// The chunk's states at every eighth token are formed first; then its batches, last to first.
template <typename Ti, typename Tu, typename Tg, bool PAIR>
__global__ void __launch_bounds__(kDirectThreads)
glr_bwd_direct_kernel(Args p, const float* __restrict__ chunk_states, const Tu* __restrict__ dh,
                      const float* __restrict__ d_state_out, Tg* __restrict__ dx,
                      Tg* __restrict__ dr, Tg* __restrict__ di, float* __restrict__ d_state_in,
                      float* __restrict__ partial) {
  const int D = p.D;
  const int seq = static_cast<int>(blockIdx.x / p.groups);
  const int c0 = static_cast<int>(blockIdx.x % p.groups) * kDirectChan;
  const int cA = c0 + (PAIR ? 2 : 1) * static_cast<int>(threadIdx.x);
  const int cB = cA + (PAIR ? 1 : kDirectThreads);
  const bool okA = cA < D, okB = cB < D;
  if (c0 == 0 && threadIdx.x == 0) check_offsets(p.L, seq, p.err);
  if (!okA) return;
  const Ti* x = static_cast<const Ti*>(p.x);
  const Ti* r = static_cast<const Ti*>(p.r);
  const Ti* i = static_cast<const Ti*>(p.i);
  int t0, t1;
  seq_bounds(p.L, seq, t0, t1);
  const F2 lm = load2(p.lam, 0, cA, cB, D);
  const F2 ysc = gate_scale(p.c, lm);
  const size_t so = static_cast<size_t>(seq) * D;
  F2 e = load2(d_state_out, so, cA, cB, D), usum = f2(0.f);
  F2 enter[kGlrChunk / kBatch];           // the state before each batch of the chunk
  for (int ch = ceil_div(t1 - t0, kGlrChunk) - 1; ch >= 0; --ch) {
    const int first = t0 + ch * kGlrChunk, end = min(first + kGlrChunk, t1);
    const int batches = ceil_div(end - first, kBatch);
    F2 st = load2(chunk_states, static_cast<size_t>(chunk_row(t0, seq) + ch) * D, cA, cB, D);
    for (int b = 0; b < batches; ++b) {
      enter[b] = st;
      if (b + 1 == batches) break;
      const size_t at = static_cast<size_t>(first + b * kBatch) * D + cA;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const size_t o = at + static_cast<size_t>(k) * D;
        F2 a, root;
        decay<false>(mul(ysc, sigmoid(load_two<Ti, PAIR>(r + o, true, okB))), a, root);
        st = fma(a, st, mul(mul(root, sigmoid(load_two<Ti, PAIR>(i + o, true, okB))),
                            load_two<Ti, PAIR>(x + o, true, okB)));
      }
    }
    for (int b = batches - 1; b >= 0; --b) {
      const int t = first + b * kBatch;
      const size_t at = static_cast<size_t>(t) * D + cA;
      F2 xv[kBatch], uv[kBatch], a[kBatch], root[kBatch], sr[kBatch], si[kBatch], hp[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool in = t + k < end;
        const size_t o = at + static_cast<size_t>(k) * D;
        xv[k] = load_two<Ti, PAIR>(x + o, in, in && okB);
        sr[k] = load_two<Ti, PAIR>(r + o, in, in && okB);
        si[k] = load_two<Ti, PAIR>(i + o, in, in && okB);
        uv[k] = load_two<Tu, PAIR>(dh + o, in, in && okB);
      }
      F2 hs = enter[b];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        sr[k] = sigmoid(sr[k]);
        si[k] = sigmoid(si[k]);
        decay<false>(mul(ysc, sr[k]), a[k], root[k]);
        hp[k] = hs;
        hs = fma(a[k], hs, mul(mul(root[k], si[k]), xv[k]));
      }
#pragma unroll
      for (int k = kBatch - 1; k >= 0; --k) {
        if (t + k >= end) continue;
        const F2 G = add(uv[k], e);
        F2 gx, gr, gi, u;
        e = mul(a[k], G);
        gate_gradients<Pairs<true>>(G, e, a[k], root[k], mul(ysc, sr[k]), sr[k], si[k], xv[k],
                                    hp[k], gx, gr, gi, u);
        usum = add(usum, u);
        const size_t o = at + static_cast<size_t>(k) * D;
        store_two<Tg, PAIR>(dx + o, gx, true, okB);
        store_two<Tg, PAIR>(dr + o, gr, true, okB);
        store_two<Tg, PAIR>(di + o, gi, true, okB);
      }
    }
  }
  if (d_state_in) store2(d_state_in, so, e, cA, cB, D);
  store2(partial, so, usum, cA, cB, D);
}

// With t = exp(-|x|): 1 / ((1 + t) (x + log1p(t))) for x > 0, t / ((1 + t) log1p(t)) otherwise, so
// that no exponential overflows.  The second tends to one as t vanishes.
__device__ __forceinline__ float sigmoid_over_softplus(float x) {
  const float t = expf(-fabsf(x));
  if (x > 0.f) return 1.0f / ((1.0f + t) * (x + log1pf(t)));
  return t == 0.f ? 1.f : t / ((1.0f + t) * log1pf(t));
}

// d_lam = (sum of the partial rows) sigmoid(lam) / softplus(lam).  32 channels
// per block; eight row groups, each in order, then the groups in order.  There is a row per sequence
// and CTA of a cluster: with very many short sequences this chain is most of the gradients' time
// (65536 x 1 x 256: 1.25 ms, the forward 0.16 ms).
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
  d_lam[d] = s * sigmoid_over_softplus(lam[d]);
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
  decay<false>(gate_scale(c, lam[d]) * sigmoid(Io<Ti>::ld(r, at)), a, root);
  const float st = fmaf(a, state[at], root * sigmoid(Io<Ti>::ld(i, at)) * Io<Ti>::ld(x, at));
  state_out[at] = st;
  if (h) Io<Th>::st(h, at, st);
}

// ---- launches --------------------------------------------------------------

template <typename F>
cudaError_t by_type(DType t, F&& f) {
  return t == DType::F32 ? f(float{}) : f(__nv_bfloat16{});
}
// The rows of every staged tensor have to allow the pieces: those of the narrowest type decide.
template <typename F>
cudaError_t by_mode(bool any_bf16, int D, F&& f) {
  const int e = any_bf16 ? 2 : 4;
  if (D * static_cast<long long>(e) % 16 == 0) return f(std::integral_constant<int, kWide>{});
  if (D % 2 == 0) return f(std::integral_constant<int, kEven>{});
  return f(std::integral_constant<int, kOdd>{});
}

// CTAs per cluster, from a model of the time in us.  A round takes a CTA about 1.4 + 0.1 S when
// it is alone on its SM, and CTAs that share one bring it to 1.2 per round of each; a cluster
// has ceil(tiles / S) rounds and about one more to start and end, and finds room the later the
// larger it is (2 % per CTA, 30 % more where clusters of sixteen share SMs).  Sizes that are not
// listed are placed badly.  Measured in us, forward / gradients: 2 x 8192 x 4096 bf16 S = 1:
// 178/296, 2: 134/266, 4: 148/271, 7: 158/324, 16: 173/360; 1 x 16384 x 1024 S = 4: 116/187,
// 8: 72/141, 12: 57/106, 14: 64/144, 16: 57/128; 1 x 1024 x 2048 S = 1: 25/41, 8: 9/15, 16: 11/21.
// Packed sequences differ in length, which the host does not know: the SMs share the sum, each
// cluster rounded up and started, while the longest, taken as four times the average, goes on
// alone (64 sequences, 200000 tokens x 1024: S = 1: 490/809, 2: 351/688, 4: 378/780, 16: 683/1391;
// 17 of 9001 x 1001 float32 S = 1: 95/154, 3: 51/79, 4: 44/82, 16: 104/195; 40 of 20000 x 2048 bf16
// S = 1: 74/140, 2: 82/181, 4: 128/242).  That is about what a uniformly cut batch has.  A batch with
// one much longer sequence gets too few CTAs for it: 8192 tokens beside 127 single ones at D = 2048
// take 192/313, alone 45/79; beside 32 at D = 4096 184/305, alone 74/180.
constexpr double kSms = 148.0;
int split_of(const SeqLayout& L, int D) {
  const double pairs = static_cast<double>((D + kChan - 1) / kChan) * L.nseq;
  const long long per = static_cast<long long>(L.nseq) * kTile;
  const long long tiles = (L.Ttot + per - 1) / per;
  int best = 1;
  double cost = 0.0;
  for (const int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
    if (s > 1 && s > tiles) break;
    const double round = 1.4 + 0.1 * s;          // us
    double c;
    if (L.T > 0) {
      const double share = std::ceil(pairs * s / kSms);
      c = static_cast<double>((tiles + s - 1) / s + 1) * std::fmax(round, 1.2 * share) *
          (0.98 + 0.02 * s) * (s == kMaxSplit && share > 1.0 ? 1.3 : 1.0);
    } else {
      const double sum = 1.2 * pairs * (static_cast<double>(tiles) + 1.5 * s) / kSms;
      const double longest = round * std::fmin(4.0, L.nseq) * static_cast<double>(tiles) / s;
      c = std::fmax(sum, longest) + 0.2 * std::fmin(sum, longest);
    }
    if (s == 1 || c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

// Whether threads walk their sequences alone: up to 32 tokens per sequence (16 on average where the
// lengths differ, which the host does not know).  Measured in us, forward / gradients, alone
// and by tiles: 256 x 4 x 4096 bf16 15 / 32 and 111 / 233, 32 x 16 x 2048 6.2 / 10 and 10.8 / 20,
// 128 x 64 x 4096 78 / 196 and 66 / 158.  A packed batch whose average is short because of many short
// sequences beside a long one loses by it, a thread walking the long one: 4096 tokens beside 300 single
// ones x 2048 919 / 1641 and 113 / 181 (alone 24 / 44), 1900 beside 127 318 / 539 and 60 / 100.
bool direct(const SeqLayout& L) {
  return L.Ttot <= (L.T > 0 ? 32ll : 16ll) * L.nseq;
}

// Launches `kern` on clusters of `split` CTAs, with `bytes` of shared memory and what the exchange
// takes (exchange_bytes of `warps` warps).  The kernel's limit belongs to the process, and other host
// threads launch between a call's setting and its launch: so every call sets the same one, that of
// the largest cluster.
template <typename... P, typename... A>
cudaError_t launch_split(void (*kern)(P...), int warps, size_t bytes, long long blocks, int split,
                         cudaStream_t s, A... args) {
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(exchange_bytes(kMaxSplit, warps) + bytes));
  if (e == cudaSuccess && split > 8)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = exchange_bytes(split, warps) + bytes;
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

long long glr_bwd_partial_rows(const SeqLayout& L, int D) {
  return static_cast<long long>(L.nseq) * (direct(L) ? 1 : split_of(L, D));
}

cudaError_t launch_glr_fwd(const void* x, const void* r, const void* i, DType in_t,
                           const float* lam, float c, const SeqLayout& L, const float* state_in,
                           float* state_out, void* h, DType h_t, float* chunk_states, int D,
                           unsigned* err, cudaStream_t s) {
  Args p{x, r, i, lam, c, L, D, (D + kChan - 1) / kChan,
         split_of(L, D), err};
  const bool alone = direct(L);
  if (alone) {
    p.groups = (D + kDirectChan - 1) / kDirectChan;
    p.split = 1;
  }
  const long long blocks = static_cast<long long>(p.groups) * L.nseq * p.split;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return by_type(in_t, [&](auto ti) {
    return by_type(h_t, [&](auto th) {
      if (alone) {
        using Ti = decltype(ti);
        using Th = decltype(th);
        auto kern = D % 2 == 0 ? glr_fwd_direct_kernel<Ti, Th, true>
                               : glr_fwd_direct_kernel<Ti, Th, false>;
        kern<<<static_cast<unsigned>(blocks), kDirectThreads, 0, s>>>(
            p, state_in, state_out, static_cast<Th*>(h), chunk_states);
        return cudaGetLastError();
      }
      return by_mode(in_t == DType::BF16, D, [&](auto mode) {
        using Ti = decltype(ti);
        using Th = decltype(th);
        constexpr int M = decltype(mode)::value;
        const size_t rows = stages<Ti>() * 3 * kFwdWarps * run_bytes<Ti, M, kFwdRun>();
        return launch_split(glr_fwd_kernel<Ti, Th, M>, kFwdWarps, rows, blocks, p.split, s, p,
                            state_in, state_out, static_cast<Th*>(h), chunk_states);
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
         split_of(L, D), err};
  const bool alone = direct(L);
  if (alone) {
    p.groups = (D + kDirectChan - 1) / kDirectChan;
    p.split = 1;
  }
  const long long blocks = static_cast<long long>(p.groups) * L.nseq * p.split;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const cudaError_t e = by_type(in_t, [&](auto ti) {
    return by_type(dh_t, [&](auto tu) {
      return by_type(g_t, [&](auto tg) {
        if (alone) {
          using Ti = decltype(ti);
          using Tu = decltype(tu);
          using Tg = decltype(tg);
          auto kern = D % 2 == 0 ? glr_bwd_direct_kernel<Ti, Tu, Tg, true>
                                 : glr_bwd_direct_kernel<Ti, Tu, Tg, false>;
          kern<<<static_cast<unsigned>(blocks), kDirectThreads, 0, s>>>(
              p, chunk_states, static_cast<const Tu*>(d_h), d_state_out, static_cast<Tg*>(dx),
              static_cast<Tg*>(dr), static_cast<Tg*>(di), d_state_in, partial);
          return cudaGetLastError();
        }
        return by_mode(in_t == DType::BF16 || dh_t == DType::BF16, D, [&](auto mode) {
          using Ti = decltype(ti);
          using Tu = decltype(tu);
          using Tg = decltype(tg);
          constexpr int M = decltype(mode)::value;
          const size_t rows = stages<Ti>() * kBwdWarps *
                              (3 * run_bytes<Ti, M, kBwdRun>() + run_bytes<Tu, M, kBwdRun>());
          const size_t states = 2 * kBwdWarps * 32 * sizeof(F2);
          return launch_split(glr_bwd_kernel<Ti, Tu, Tg, M>, kBwdWarps, states + rows, blocks,
                              p.split, s, p, chunk_states, static_cast<const Tu*>(d_h), d_state_out,
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
