// rlk_sampling.cu -- what a rollout does with a row of logits: probabilities
// at the row's temperature, and the verification of drafted tokens against the
// target's probabilities from given random numbers.
//
// Both are bound by the one pass over the rows they read (and, for the
// probabilities, write), or at few rows by latency.  A row is the work of one
// thread-block cluster.  Every sum takes the entries by their place in the row, in
// an order that depends on V and the type only: not on how many rows there are, on
// where the row sits, or on its alignment (an odd V puts every row at another
// offset within 16 bytes).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rlk.h"
#include "rlk_device.h"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

constexpr size_t kSampHeader = 256;  // word 0: the device error word
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kSampLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store_as(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A CTA may write another's shared memory once that one runs: each arrives
// when it starts and waits for the others just before its first such write.
__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_all_started() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// =====================================================================
// probabilities
// =====================================================================

// p[v] = 2^((x[v] - m) k) / S,  k = log2(e) / tau,  m = max x,  S = sum of the
// numerators; tau = 0 puts 1 at the first maximum.
//
// A row belongs to a cluster of 1, 2, 4 or 8 CTAs, by V and the type alone: the
// fewest whose shared memory holds it at two CTAs per SM.  A CTA copies its slice
// in (16-byte asynchronous copies; a slice that starts off a 16-byte boundary sits
// as far off in shared memory) and looks at it three times: its maximum, its sum
// relative to that, and, when the slices' pairs (maximum, sum) have met, the
// probabilities.  The sum takes entries by their place in the slice, whatever the
// slice's alignment, so its order is the same for every row; the other two looks
// take whole aligned vectors.
//
// Each entry is read once and written once, one CTA's copies running beside another's
// looks.  320 x 151936 fp32: 74 us, 0.80 of the measured copy, bound by HBM; bf16 to
// fp32 55 us, 0.81.  With fewer bytes per entry the looks weigh more, and neither HBM
// nor issue is full: 1027 x 50257 bf16 45 us, HBM 0.70, issue slots 0.42; two CTAs per
// SM, and each waits for all of its copies before its first look, so one CTA's looks are
// all that covers the other's copies.  Where the types differ the stores are single
// entries: fp32 to bf16 67 us at 320 x 151936, 0.66.  One row of 151936: 6.6 us.
// Holding the entries in registers (one look, one exponential, but 64 warps to a row of
// 50257, each with its reductions) ran 55 instructions per entry and 128 us at
// 1027 x 50257.  Persistent CTAs with the same three looks took 94 us at 320 x 151936
// and 54 at 1027 x 50257; 512 threads 91 and 46, 128 threads 84 and 54.
//
// Precision, of fp32 results: the factor k, each exponent, ex2.approx (2^-22),
// 1 / S and the product are rounded to fp32, so an entry D powers of two
// below the maximum is off by up to (3 D + 10) 2^-24 relative; in the norm 1.1e-7 from
// fp64 at the measured cases, where expf and a division give 6e-8.  Splitting k or a
// longer exponential would cost an instruction or more per entry and look; the
// verification that follows compares with random numbers of 24 bits.
constexpr int kProbMaxCluster = 8;
constexpr int kProbThreads = 256;
constexpr uint32_t kProbSlice = 100u * 1024u;  // bytes of a slice at most
constexpr uint32_t kProbPad = 48u;             // room for an offset and whole vectors behind

struct ProbArgs {
  const void* x;
  void* p;
  const float* row_tau;
  int64_t ldx, ldp;
  int64_t R;
  int V;
  int slice;  // entries per CTA of the cluster
  float tau;
  unsigned* err;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// What every warp folds from the pairs of a long row: its maximum and S (or, greedy,
// the least index of the maximum).
struct RowStats {
  float m, S;
  int at;
  bool nan;
};

__device__ __forceinline__ RowStats fold_pairs(const uint2* pairs, int n, float k, bool greedy,
                                               int lane) {
  RowStats r{-INFINITY, 0.f, INT_MAX, false};
  for (int i = lane; i < n; i += 32) {
    const float mi = __uint_as_float(pairs[i].x);
    r.m = fmaxf(r.m, mi);
    r.nan |= mi != mi;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.m = fmaxf(r.m, __shfl_xor_sync(kFull, r.m, o));
  if (greedy) {
    r.nan = __any_sync(kFull, r.nan);
    for (int i = lane; i < n; i += 32)
      if (__uint_as_float(pairs[i].x) == r.m) r.at = min(r.at, static_cast<int>(pairs[i].y));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r.at = min(r.at, __shfl_xor_sync(kFull, r.at, o));
    return r;
  }
  const float ref = r.m == -INFINITY ? 0.f : r.m;  // -inf - -inf would be NaN
  for (int i = lane; i < n; i += 32)
    r.S += __uint_as_float(pairs[i].y) * ex2_approx((__uint_as_float(pairs[i].x) - ref) * k);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.S += __shfl_xor_sync(kFull, r.S, o);
  return r;
}

// A row's probabilities from its logits; greedy rows are `inv` (0 or NaN) but at
// one place.
struct RowOut {
  float ref, k, inv;
  int at;  // greedy: where the one is (-1: nowhere)
  __device__ __forceinline__ float operator()(float x) const { return ex2_approx((x - ref) * k) * inv; }
  __device__ __forceinline__ float at_place(int i) const { return i == at ? 1.f : inv; }
};

// Sets `bad` where the row gives no distribution: nothing left by its mask
// (zeros), or a NaN, +inf, or a temperature that is not a positive finite number
// (NaN).
__device__ __forceinline__ RowOut row_out(const RowStats& r, float tau, float k, bool greedy,
                                          bool& bad) {
  RowOut o;
  o.k = k;
  o.ref = r.m == -INFINITY ? 0.f : r.m;
  const bool empty = r.m == -INFINITY;
  const bool usable = greedy ? !r.nan : tau > 0.f && k > 0.f && k < INFINITY && r.S == r.S;
  o.inv = !usable ? NAN : empty || greedy ? 0.f : 1.f / r.S;
  o.at = empty || !usable ? -1 : r.at;
  bad = !usable || empty;
  return o;
}

// A maximum's numerators: 2^(x k - c) with c = ref k as rounded, one operation per
// entry.  The rounding of c, d = ref k - c, is common to all numerators and to their
// sum and cancels between them; where |c| is so large that 2^d would matter on its
// own (d reaches 2^-24 |c|), 2^((x - ref) k) instead.
struct RowExp {
  float k, ref, c;
  bool plain;
  __device__ __forceinline__ RowExp(float m, float kk) {
    k = kk;
    ref = m == -INFINITY ? 0.f : m;  // -inf - -inf would be NaN
    c = ref * k;
    plain = fabsf(c) < 1e6f;
  }
  // the factor that takes this one's numerators to another's
  __device__ __forceinline__ float shift(const RowExp& to) const {
    if (plain && to.plain) return ex2_approx(c - to.c);
    float e = (ref - to.ref) * k;
    if (plain) e -= fmaf(ref, k, -c);
    if (to.plain) e += fmaf(to.ref, k, -to.c);
    return ex2_approx(e);
  }
};

template <typename T, int kThreads>
struct Slice {
  static constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // entries per 16 bytes
  static constexpr int kPair = sizeof(T) == 2 ? 2 : 1;
  // largest entry of `nv` aligned vectors
  static __device__ __forceinline__ float maximum(const T* room, int nv) {
    const uint4* src = reinterpret_cast<const uint4*>(room);
    if constexpr (kPair == 1) {
      float m = -INFINITY;
#pragma unroll 4
      for (int i = threadIdx.x; i < nv; i += kThreads) {
        const uint4 q = src[i];
        m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(q.x), __uint_as_float(q.y))),
                  fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
      }
      return m;
    } else {
      __nv_bfloat162 m = __floats2bfloat162_rn(-INFINITY, -INFINITY);
#pragma unroll 4
      for (int i = threadIdx.x; i < nv; i += kThreads) {
        const uint4 q = src[i];
        const __nv_bfloat162 a = __hmax2(as2(q.x), as2(q.y)), b = __hmax2(as2(q.z), as2(q.w));
        m = __hmax2(m, __hmax2(a, b));
      }
      return fmaxf(__low2float(m), __high2float(m));
    }
  }
  // sum of f over the n entries at buf = room + off, by their place
  template <typename F>
  static __device__ __forceinline__ float sum(const T* buf, int off, int n, F f) {
    float s = 0.f;
    if constexpr (kPair == 1) {
#pragma unroll 8
      for (int i = threadIdx.x; i < n; i += kThreads) s += f(to_f32(buf[i]));
    } else {
      // pairs of neighbours; at an odd offset a pair straddles two words
      const int np = (n + 1) >> 1;  // the entry behind an odd n is -inf
      const uint32_t* w = reinterpret_cast<const uint32_t*>(buf - (off & 1));
      if (off & 1) {
#pragma unroll 8
        for (int i = threadIdx.x; i < np; i += kThreads)
          s = add(s, __funnelshift_r(w[i], w[i + 1], 16), f);
      } else {
#pragma unroll 8
        for (int i = threadIdx.x; i < np; i += kThreads) s = add(s, w[i], f);
      }
    }
    return s;
  }
  template <typename F>
  static __device__ __forceinline__ float add(float s, uint32_t x, F f) {
    s += f(__uint_as_float(x << 16));
    return s + f(__uint_as_float(x & 0xffff0000u));
  }
  static __device__ __forceinline__ __nv_bfloat162 as2(uint32_t u) {
    return *reinterpret_cast<const __nv_bfloat162*>(&u);
  }
  // p = f of the n entries
  template <typename TOut, typename F>
  static __device__ __forceinline__ void write(TOut* p, const T* room, int off, int n, F f) {
    const T* buf = room + off;
    if (sizeof(T) == sizeof(TOut) &&
        (reinterpret_cast<uintptr_t>(p) & 15u) == off * sizeof(T)) {
      // the same place within 16 bytes: whole vectors, but at the ends
      const int head = min(n, (kVec - off) & (kVec - 1));
      const int nv = (n - head) / kVec;
      const uint4* src = reinterpret_cast<const uint4*>(buf + head);
      uint4* dst = reinterpret_cast<uint4*>(p + head);
#pragma unroll 4
      for (int i = threadIdx.x; i < nv; i += kThreads) {
        const uint4 q = src[i];
        dst[i] = make_uint4(word(q.x, f), word(q.y, f), word(q.z, f), word(q.w, f));
      }
      const int t = threadIdx.x, tail = head + nv * kVec;
      if (t < head) store_as(p + t, f(to_f32(buf[t])));
      if (t < n - tail) store_as(p + tail + t, f(to_f32(buf[tail + t])));
    } else {
#pragma unroll 8
      for (int i = threadIdx.x; i < n; i += kThreads) store_as(p + i, f(to_f32(buf[i])));
    }
  }
  template <typename F>
  static __device__ __forceinline__ uint32_t word(uint32_t x, F f) {
    if constexpr (kPair == 1) {
      return __float_as_uint(f(__uint_as_float(x)));
    } else {
      const __nv_bfloat162 b =
          __floats2bfloat162_rn(f(__uint_as_float(x << 16)), f(__uint_as_float(x & 0xffff0000u)));
      return *reinterpret_cast<const uint32_t*>(&b);
    }
  }
};

template <typename TIn, typename TOut, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 128 ? 8 : 4) probs_kernel(const ProbArgs P) {
  using S = Slice<TIn, kThreads>;
  constexpr int kWarps = kThreads / 32;
  constexpr int kVec = S::kVec;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float warp_max[kWarps], warp_sum[kWarps];
  __shared__ int warp_at[kWarps];
  __shared__ uint2 met[kProbMaxCluster];
  TIn* room = reinterpret_cast<TIn*>(smem);
  uint32_t C, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  if (C > 1) cluster_started();
  const int64_t row = blockIdx.x / C;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int lo = static_cast<int>(min(static_cast<int64_t>(rank) * P.slice, static_cast<int64_t>(P.V)));
  const int n = min(P.slice, P.V - lo);  // this CTA's entries
  // the slice, and -inf around it up to whole vectors
  const TIn* g = static_cast<const TIn*>(P.x) + row * P.ldx + lo;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(TIn));
  const int nv = (off + n + kVec) / kVec;  // vectors, one entry more than the slice at least
  {
    const int head = min(n, (kVec - off) & (kVec - 1));
    const int whole = (n - head) / kVec;
    const uint32_t dst = smem_u32(room + off + head);
    for (int i = t; i < whole; i += kThreads) cp_async16(dst + i * 16, g + head + i * kVec);
    const int tail = head + whole * kVec;
    if (t < head) room[off + t] = g[t];
    if (t < n - tail) room[off + tail + t] = g[tail + t];
    if (t < off) store_as(room + t, -INFINITY);
    if (t < nv * kVec - off - n) store_as(room + off + n + t, -INFINITY);
  }
  const float tau = P.row_tau ? P.row_tau[row] : P.tau;
  const float k = kSampLog2e / tau;
  const bool greedy = tau == 0.f;
  cp_async_wait_all();
  __syncthreads();

  float m = S::maximum(room, nv);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  if (lane == 0) warp_max[warp] = m;
  __syncthreads();
  m = warp_max[lane & (kWarps - 1)];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));

  const RowExp e(m, k);
  const TIn* buf = room + off;
  float s = 0.f;
  int at = INT_MAX;
  if (greedy) {  // the first maximum; a NaN makes the sum one
    for (int i = t; i < n; i += kThreads) {
      const float x = to_f32(buf[i]);
      if (x != x) s = NAN;
      if (x == m) at = min(at, lo + i);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) at = min(at, __shfl_xor_sync(kFull, at, o));
    if (lane == 0) warp_at[warp] = at;
  } else if (e.plain) {
    s = S::sum(buf, off, n, [&](float x) { return ex2_approx(fmaf(x, e.k, -e.c)); });
  } else {
    s = S::sum(buf, off, n, [&](float x) { return ex2_approx((x - e.ref) * e.k); });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
  if (lane == 0) warp_sum[warp] = s;
  __syncthreads();
  s = warp_sum[lane & (kWarps - 1)];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
  if (greedy) {
    at = warp_at[lane & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) at = min(at, __shfl_xor_sync(kFull, at, o));
  }
  if (C > 1) {
    // the slices' maxima and sums (or, greedy, the places; NaN as the maximum)
    cluster_all_started();
    if (warp == 0 && lane < C)
      st_cluster_v2(mapa_shared(smem_u32(&met[rank]), lane),
                    __float_as_uint(greedy && s != s ? NAN : m),
                    greedy ? static_cast<uint32_t>(at) : __float_as_uint(s));
    cluster_sync();
    float gm = -INFINITY;
    for (int i = 0; i < static_cast<int>(C); ++i) gm = fmaxf(gm, __uint_as_float(met[i].x));
    const RowExp all(gm, k);
    s = 0.f;
    at = INT_MAX;
    for (int i = 0; i < static_cast<int>(C); ++i) {
      const float mi = __uint_as_float(met[i].x);
      if (greedy) {
        if (mi != mi) s = NAN;
        if (mi == gm) at = min(at, static_cast<int>(met[i].y));
      } else if (mi != -INFINITY || __uint_as_float(met[i].y) != 0.f) {
        s += __uint_as_float(met[i].y) * RowExp(mi, k).shift(all);
      }
    }
    m = gm;
  }

  // a row that gives no distribution: nothing left by its mask (zeros), or a NaN,
  // +inf, or a temperature that is not a positive finite number (NaN)
  const bool usable = s == s && (greedy || (tau > 0.f && k > 0.f && k < INFINITY));
  const bool empty = m == -INFINITY;
  if ((!usable || empty) && rank == 0 && t == 0) atomicOr(P.err, RLK_DEVERR_PROBS);
  TOut* p = static_cast<TOut*>(P.p) + row * P.ldp + lo;
  if (!usable || empty || greedy) {
    const float rest = usable ? 0.f : NAN;
    if (!usable || empty) at = -1;
#pragma unroll 8
    for (int i = t; i < n; i += kThreads) store_as(p + i, lo + i == at ? 1.f : rest);
  } else {
    const RowExp o(m, k);
    const float inv = 1.f / s;
    if (o.plain) {
      S::write(p, room, off, n, [&](float x) { return ex2_approx(fmaf(x, o.k, -o.c)) * inv; });
    } else {
      S::write(p, room, off, n, [&](float x) { return ex2_approx((x - o.ref) * o.k) * inv; });
    }
  }
}

// Rows that no cluster's shared memory holds (more than 204800 entries in fp32, 409600
// in bf16): one CTA per row and eighth, its entries read again from L2 or HBM for the
// second and third look, one at a time.  262144 fp32: one row 17 us, 320 rows 206 us (0.50
// of the measured copy, where 320 rows of 204800 take 108, 0.74); 409601 bf16: 28 and
// 287 us (0.28).
constexpr int kProbLongThreads = 512;
constexpr int kProbLongWarps = kProbLongThreads / 32;

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kProbLongThreads) probs_long_kernel(const ProbArgs P) {
  __shared__ uint2 pairs[kProbMaxCluster * kProbLongWarps];
  uint32_t C, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  cluster_started();
  const int64_t row = blockIdx.x / C;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int lo = static_cast<int>(min(static_cast<int64_t>(rank) * P.slice, static_cast<int64_t>(P.V)));
  const int n = min(P.slice, P.V - lo);
  const TIn* x = static_cast<const TIn*>(P.x) + row * P.ldx + lo;
  TOut* p = static_cast<TOut*>(P.p) + row * P.ldp + lo;
  const float tau = P.row_tau ? P.row_tau[row] : P.tau;
  const float k = kSampLog2e / tau;
  const bool greedy = tau == 0.f;
  float m = -INFINITY;
#pragma unroll 16
  for (int i = t; i < n; i += kProbLongThreads) m = fmaxf(m, to_f32(x[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  uint2 mine;
  if (greedy) {
    int first = INT_MAX;
    bool nan = false;
#pragma unroll 16
    for (int i = t; i < n; i += kProbLongThreads) {
      const float v = to_f32(x[i]);
      nan |= v != v;
      if (v == m) first = min(first, lo + i);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first = min(first, __shfl_xor_sync(kFull, first, o));
    if (__any_sync(kFull, nan)) m = NAN;
    mine = make_uint2(__float_as_uint(m), static_cast<uint32_t>(first));
  } else {
    float s = 0.f;
#pragma unroll 16
    for (int i = t; i < n; i += kProbLongThreads) s += ex2_approx((to_f32(x[i]) - ref) * k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    mine = make_uint2(__float_as_uint(m), __float_as_uint(s));
  }
  cluster_all_started();
  if (lane < C)
    st_cluster_v2(mapa_shared(smem_u32(&pairs[rank * kProbLongWarps + warp]), lane), mine.x, mine.y);
  cluster_sync();
  const RowStats rs = fold_pairs(pairs, static_cast<int>(C) * kProbLongWarps, k, greedy, lane);
  bool bad;
  const RowOut out = row_out(rs, tau, k, greedy, bad);
  if (bad && rank == 0 && t == 0) atomicOr(P.err, RLK_DEVERR_PROBS);
#pragma unroll 16
  for (int i = t; i < n; i += kProbLongThreads)
    store_as(p + i, greedy ? out.at_place(lo + i) : out(to_f32(x[i])));
}

// =====================================================================
// verification of drafted tokens
// =====================================================================

// For sequence b with draft tokens d_0 .. d_{len-1}:
//   n      = the first i with not (ua_i q_i(d_i) < p_i(d_i)), len if none
//   r(v)   = max(0, p_n(v) - q_n(v)) if n < len, p_n(v) if n = len
//            (p_n too where that residual is zero everywhere)
//   token  = the least v with r(0) + .. + r(v) > us (r(0) + .. + r(V - 1))
// Products, differences and sums are in 64 bits: an fp32 product is exact
// there, and the running sum of a vocabulary keeps the borders between
// tokens where the probabilities put them (in 32 bits they would move by more
// than the smallest probabilities).
//
// The vocabulary is cut into at most kVerMaxSegs segments whose length follows
// from V alone (256 entries up to V = 163840).  A warp sums a segment in a fixed
// order, the totals meet in every CTA of the sequence's cluster, every warp finds
// the segment that the threshold falls in by the same running sum, and the warp
// that summed it walks it once more (from L2).  So a token does not depend on the
// cluster's size, which follows the number of sequences.
//
// Bound by latency at few sequences (the drafts, their entries, the row, the
// walk: four round trips and a cluster barrier): one of 4 drafts and V = 151936 7.6 us.
// At many in fp32, by HBM once those are over: 64 sequences 19.5 us, 78 MB of rows in 11
// of them.  In bf16 by instructions and latency together: 256 ragged sequences of V =
// 50257 24.6 us against 7.9 of bytes; 10.8 M warp instructions, 27 per 32 entries of a
// row (p and q), come to 11 us of issue on the SMs that hold two of the 256 CTAs
// (issuing in 63% of their active cycles), the rest is loads waited for and the fixed
// trips; 256 rows of 151936 50 us, 3.1 TB/s, 24.8 M instructions, 68%.  What did not
// help: copies through shared memory ahead of the sums (26 us at 64), several segments'
// loads at once or the next one's ahead in registers (21), 256 threads (19.1, but 9.3 at
// one).
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerMaxCluster = 8;
constexpr int kVerPiece = 256;      // entries walked at a time: 8 consecutive ones per lane
constexpr int kVerPer = 20;         // segments per lane of the running sum
constexpr int kVerMaxSegs = 32 * kVerPer;

struct VerifyArgs {
  const void* p;
  const void* q;  // null: the draft has probability one at its own token
  int64_t p_sb, p_sk, q_sb, q_sk;
  const int64_t* drafts;
  const float* ua;
  const float* us;
  const int64_t* lens;
  int64_t K;
  int V;
  int seg;   // entries per segment, a multiple of kVerPiece
  int nseg;
  int64_t* tokens;
  int64_t* accepted;
  unsigned* err;
};

// x 2^-896 in 64 bits, exactly: the exponent's field moved, not rebiased (a shift
// and a mask, where converting takes the slow path of the conversion unit; zeros
// and subnormals come out right by themselves).  Sums of such values, and their
// comparison with a share of their own sum, need no scaling back.
template <typename T>
__device__ __forceinline__ double scaled(float x) {
  const int u = __float_as_int(x);
  // a bf16 has no bits that reach the lower word
  return __hiloint2double((u >> 3) & static_cast<int>(0x8fffffffu), sizeof(T) == 2 ? 0 : u << 29);
}

// max(0, p - q), scaled; `taint` becomes NaN where either is NaN or infinite.
template <typename T>
__device__ __forceinline__ double residual(float p, float q, float& taint) {
  taint = fmaf(p, 0.f, fmaf(q, 0.f, taint));
  return scaled<T>(fmaxf(p, q)) - scaled<T>(q);
}

// The index in a 256-entry piece of a lane's entry j: one by one in fp32, pairs of
// neighbours in bf16.
template <typename T>
__device__ __forceinline__ int piece_index(int lane, int j) {
  return sizeof(T) == 4 ? lane + 32 * j : 2 * lane + 64 * (j >> 1) + (j & 1);
}

// A lane's 8 entries of the piece at `row`, all of it inside the row.  kOdd: a bf16
// piece that starts off a word's boundary; each pair is put together from two lanes'
// words, and nothing outside the piece but the entry before it, in the same word,
// is read (`begins`: not even that, the row begins here).
template <bool kOdd>
__device__ __forceinline__ void load_piece(float (&v)[8], const float* row, bool, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = row[lane + 32 * j];
}
template <bool kOdd>
__device__ __forceinline__ void load_piece(float (&v)[8], const __nv_bfloat16* row, bool begins,
                                           int lane) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
  const uint32_t* x = reinterpret_cast<const uint32_t*>(h - (kOdd ? 1 : 0)) + lane;
  uint32_t w[4], behind = 0u;
  if constexpr (kOdd) {
    const bool lone = begins && lane == 0;
    w[0] = lone ? static_cast<uint32_t>(h[0]) << 16 : x[0];
    if (lane == 0) behind = h[kVerPiece - 1];
  } else {
    w[0] = x[0];
  }
#pragma unroll
  for (int j = 1; j < 4; ++j) w[j] = x[32 * j];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t two = w[j];
    if constexpr (kOdd) {  // lane 31 goes on in lane 0's next word
      const uint32_t give = lane == 0 ? (j < 3 ? w[j < 3 ? j + 1 : 3] : behind) : w[j];
      two = __funnelshift_r(two, __shfl_sync(kFull, give, (lane + 1) & 31), 16);
    }
    v[2 * j] = __uint_as_float(two << 16);
    v[2 * j + 1] = __uint_as_float(two & 0xffff0000u);
  }
}

__device__ __forceinline__ double tree8(const double (&r)[8]) {
  return ((r[0] + r[1]) + (r[2] + r[3])) + ((r[4] + r[5]) + (r[6] + r[7]));
}

// A lane's part of the residual's sum over one whole segment; kQ: there is a q.
// The alignment and q are the row's: the loop over segments is compiled for each
// kind, with no condition left inside (as conditions they took 40 instructions
// per entry instead of 15).
template <typename T, bool kQ, bool kOddP, bool kOddQ>
__device__ __forceinline__ double segment_part(const T* p, const T* q, int lo, int seg, int lane,
                                               float& taint) {
  double acc = 0.;
  for (int o = lo; o < lo + seg; o += kVerPiece) {
    float pv[8], qv[8];
    load_piece<kOddP>(pv, p + o, o == 0, lane);
    if constexpr (kQ) load_piece<kOddQ>(qv, q + o, o == 0, lane);
    double r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = residual<T>(pv[j], kQ ? qv[j] : 0.f, taint);
    acc += tree8(r);
  }
  return acc;
}

// The same for any segment: cut off by the row's end, or with the place where q is
// one in it.
template <typename T>
__device__ __forceinline__ double any_segment_part(const T* p, const T* q, int hot, int V, int lo,
                                                   int seg, int lane, float& taint) {
  double acc = 0.;
  for (int o = 0; o < seg; o += kVerPiece) {
    double r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = o + piece_index<T>(lane, j);
      const bool in = at < V - lo;
      const float pv = in ? to_f32(p[lo + at]) : 0.f;
      const float qv = in && q ? to_f32(q[lo + at]) : in && lo + at == hot ? 1.f : 0.f;
      r[j] = residual<T>(pv, qv, taint);
    }
    acc += tree8(r);
  }
  return acc;
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads, 1024 / kVerThreads) verify_kernel(const VerifyArgs P) {
  __shared__ __align__(16) double totals[2][kVerMaxSegs];
  __shared__ int s_n;
  uint32_t C, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  cluster_started();
  const int64_t b = blockIdx.x / C;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* pb = static_cast<const T*>(P.p) + b * P.p_sb;
  const T* qb = static_cast<const T*>(P.q) + (P.q ? b * P.q_sb : 0);
  const int64_t* drafts = P.drafts + b * P.K;
  const int V = P.V;
  const float us = P.us[b];
  int64_t len = P.lens ? P.lens[b] : P.K;
  len = len < 0 ? 0 : len > P.K ? P.K : len;

  if (warp == 0) {  // the acceptance tests, 32 drafts at a time
    int n = static_cast<int>(len);
    bool outside = false;
    for (int64_t k0 = 0; k0 < P.K; k0 += 32) {
      const int64_t k = k0 + lane;
      // what lies behind the length is loaded (it is there) but not looked at
      const int64_t d = k < P.K ? drafts[k] : 0;
      const double u = k < P.K ? P.ua[b * P.K + k] : 0.f;
      bool ok = k >= len;
      if (!ok && d >= 0 && d < V) {
        const double pd = to_f32(pb[k * P.p_sk + d]);
        const double qd = P.q ? static_cast<double>(to_f32(qb[k * P.q_sk + d])) : 1.;
        ok = u * qd < pd;
      } else {
        outside |= !ok;
      }
      const uint32_t no = __ballot_sync(kFull, !ok);
      if (no && n == static_cast<int>(len)) n = static_cast<int>(k0) + __ffs(no) - 1;
      if (rank == 0 && k < P.K && k < n) P.tokens[b * (P.K + 1) + k] = d;
    }
    if (__any_sync(kFull, outside) && lane == 0 && rank == 0) atomicOr(P.err, RLK_DEVERR_TARGET);
    if (lane == 0) s_n = n;
  } else {
    for (int i = P.nseg + threadIdx.x - 32; i < kVerMaxSegs; i += kVerThreads - 32)
      totals[0][i] = totals[1][i] = 0.;
  }
  __syncthreads();
  const int n = s_n;
  if (warp == 1 && rank == 0) {
    for (int64_t k = n + 1 + lane; k <= P.K; k += 32) P.tokens[b * (P.K + 1) + k] = -1;
    if (lane == 0) P.accepted[b] = n;
  }
  const T* p = pb + n * P.p_sk;
  const T* q = n < len && P.q ? qb + n * P.q_sk : nullptr;
  // where q is one; a draft outside [0, V) is nowhere
  const int64_t drafted = n < len && !P.q ? drafts[n] : -1;
  int hot = drafted >= 0 && drafted < V ? static_cast<int>(drafted) : -1;
  const int nw = static_cast<int>(C) * kVerWarps;
  const int my = static_cast<int>(rank) * kVerWarps + warp;  // segments my, my + nw, ...

  for (int attempt = 0;; ++attempt) {
    float taint = 0.f;
    if (attempt == 0) cluster_all_started();
    auto put = [&](int s, double acc) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
      if (__any_sync(kFull, taint != 0.f)) acc = static_cast<double>(NAN);  // no distribution
      if (lane < C)
        st_cluster_v2(mapa_shared(smem_u32(&totals[attempt][s]), lane),
                      static_cast<uint32_t>(__double2loint(acc)),
                      static_cast<uint32_t>(__double2hiint(acc)));
    };
    const int whole = V / P.seg;
    const int hot_seg = hot >= 0 ? hot / P.seg : -1;
    auto sums = [&](auto kq, auto kp, auto kr) {
      for (int s = my; s < whole; s += nw) {
        put(s, kq.value || s != hot_seg
                   ? segment_part<T, kq.value, kp.value, kr.value>(p, q, s * P.seg, P.seg, lane, taint)
                   : any_segment_part(p, q, hot, V, s * P.seg, P.seg, lane, taint));
      }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    const bool odd_p = sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(p) & 2u) != 0;
    const bool odd_q = sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(q) & 2u) != 0;
    if (!q) {
      odd_p ? sums(No{}, Yes{}, No{}) : sums(No{}, No{}, No{});
    } else if (odd_p) {
      odd_q ? sums(Yes{}, Yes{}, Yes{}) : sums(Yes{}, Yes{}, No{});
    } else {
      odd_q ? sums(Yes{}, No{}, Yes{}) : sums(Yes{}, No{}, No{});
    }
    if (whole < P.nseg && whole % nw == my)  // the row's end
      put(whole, any_segment_part(p, q, hot, V, whole * P.seg, P.seg, lane, taint));
    cluster_sync();

    // every warp: the running sum over lanes' segments, kVerPer of them per lane
    const double* tot = totals[attempt] + lane * kVerPer;
    double t[kVerPer / 2];
#pragma unroll
    for (int j = 0; j < kVerPer / 2; ++j) {
      const double2 two = *reinterpret_cast<const double2*>(tot + 2 * j);
      t[j] = two.x + two.y;
    }
#pragma unroll
    for (int j = 0; j < kVerPer / 4; ++j) t[j] += t[j + kVerPer / 4];
    const double own = (t[0] + t[1]) + (t[2] + t[3]) + t[4];
    static_assert(kVerPer == 20, "the sum above");
    double incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    const double S = __shfl_sync(kFull, incl, 31);
    if (S == 0. && attempt == 0 && n < len) {  // p <= q everywhere: take p
      q = nullptr;
      hot = -1;
      continue;
    }
    if (!(S > 0.)) {
      if (rank == 0 && threadIdx.x == 0) {
        P.tokens[b * (P.K + 1) + n] = -1;
        atomicOr(P.err, RLK_DEVERR_PROBS);
      }
      return;  // every warp of the cluster alike
    }
    // the lane, then its segment, in which the running sum passes c; the last of
    // positive residual for us >= 1 (or NaN), or should rounding leave none
    const double c = us < 1.f ? static_cast<double>(us) * S : static_cast<double>(INFINITY);
    auto first_or_last = [&](bool over, bool positive) {
      const uint32_t first = __ballot_sync(kFull, over && positive);
      const uint32_t any = __ballot_sync(kFull, positive);
      return first ? __ffs(first) - 1 : 31 - __clz(any);
    };
    const int l = first_or_last(incl > c, own > 0.);
    double before = __shfl_up_sync(kFull, incl, 1);
    before = l == 0 ? 0. : __shfl_sync(kFull, before, l);
    const double x = lane < kVerPer ? totals[attempt][l * kVerPer + lane] : 0.;
    double in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(kFull, in, o);
      if (lane >= o) in += up;
    }
    const int j = first_or_last(before + in > c, x > 0.);
    const double upto = __shfl_sync(kFull, in, (j + 31) & 31);  // of the segment before
    if (j > 0) before += upto;
    const int found = l * kVerPer + j;
    if (found % nw != my) return;

    // the segment's warp walks it, 8 consecutive entries per lane
    const int lo = found * P.seg, size = min(P.seg, V - lo);
    int token = -1;
    bool sure = false;
    for (int o = 0; o < size && !sure; o += kVerPiece) {
      const int i = lo + o + lane * 8, left = size - o - lane * 8;
      double w[8];
      float pv[8], qv[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) pv[k] = k < left ? to_f32(p[i + k]) : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        qv[k] = k < left && q ? to_f32(q[i + k]) : i + k == hot ? 1.f : 0.f;
      int last = -1;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double r = residual<T>(pv[k], qv[k], taint);
        if (r > 0.) last = k;
        w[k] = k == 0 ? r : w[k > 0 ? k - 1 : 0] + r;
      }
      double sum = w[7];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double up = __shfl_up_sync(kFull, sum, d);
        if (lane >= d) sum += up;
      }
      double base = __shfl_up_sync(kFull, sum, 1);
      base = before + (lane == 0 ? 0. : base);
      const uint32_t cross = __ballot_sync(kFull, last >= 0 && before + sum > c);
      const uint32_t pos = __ballot_sync(kFull, last >= 0);
      if (pos) {
        sure = cross != 0;
        const int at_lane = sure ? __ffs(cross) - 1 : 31 - __clz(pos);
        int at = last;
        if (sure) {
#pragma unroll
          for (int k = 7; k >= 0; --k)
            if (w[k] > (k > 0 ? w[k > 0 ? k - 1 : 0] : 0.) && base + w[k] > c) at = k;
        }
        token = lo + o + at_lane * 8 + __shfl_sync(kFull, at, at_lane);
      }
      before += __shfl_sync(kFull, sum, 31);
    }
    if (lane == 0) P.tokens[b * (P.K + 1) + n] = token;
    return;
  }
}

bool al(const void* p, uintptr_t m) { return reinterpret_cast<uintptr_t>(p) % m == 0; }

template <typename Args>
rlk_status launch_clusters(void (*kern)(Args), const Args& a, int64_t groups, int C, int threads,
                           cudaStream_t st, size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(static_cast<unsigned>(groups * C));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
    cudaGetLastError();
    return RLK_ERR_CUDA;
  }
  return RLK_OK;
}

template <typename TIn, typename TOut, int kThreads>
rlk_status launch_probs_as(const ProbArgs& a, int C, cudaStream_t st) {
  auto kern = probs_kernel<TIn, TOut, kThreads>;
  const size_t smem = static_cast<size_t>(a.slice) * sizeof(TIn) + kProbPad;
  // The limit is raised by every call that needs it (past 48 KB, less what the kernel
  // holds statically), not once: it is a fact of the context, and goes with it when the
  // device is reset.
  if (smem > 40u * 1024u &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kProbSlice + kProbPad)) != cudaSuccess) {
    cudaGetLastError();
    return RLK_ERR_CUDA;
  }
  return launch_clusters(kern, a, a.R, C, kThreads, st, smem);
}

template <typename TIn, typename TOut>
rlk_status launch_probs(ProbArgs a, cudaStream_t st) {
  constexpr int kMost = static_cast<int>(kProbSlice / sizeof(TIn));
  int C = 1;
  while (C < kProbMaxCluster && a.V > C * kMost) C *= 2;
  a.slice = (a.V - 1) / C / 32 * 32 + 32;  // V / C rounded up to whole warps
  if (a.slice > kMost)
    return launch_clusters(probs_long_kernel<TIn, TOut>, a, a.R, C, kProbLongThreads, st);
  // short rows: small CTAs, more of them per SM
  return a.V <= 2048 ? launch_probs_as<TIn, TOut, 128>(a, C, st)
                     : launch_probs_as<TIn, TOut, kProbThreads>(a, C, st);
}

}  // namespace
}  // namespace rlk

using namespace rlk;

extern "C" size_t rlk_sampling_workspace_bytes(void) { return kSampHeader; }

extern "C" rlk_status rlk_token_probs(const void* logits, int logits_type, int64_t R, int64_t V,
                                      int64_t ld_logits, float temperature,
                                      const float* row_temperature, void* probs, int probs_type,
                                      int64_t ld_probs, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (R < 0 || V <= 0 || ld_logits < V || ld_probs < V) return RLK_ERR_INVALID_ARG;
  if ((logits_type != RLK_TYPE_BF16 && logits_type != RLK_TYPE_F32) ||
      (probs_type != RLK_TYPE_BF16 && probs_type != RLK_TYPE_F32))
    return RLK_ERR_INVALID_ARG;
  if (!row_temperature && (!(temperature >= 0.f) || !std::isfinite(temperature) ||
                           (temperature > 0.f && !std::isfinite(kSampLog2e / temperature))))
    return RLK_ERR_INVALID_ARG;
  if (V >= (int64_t{1} << 31) || R > ((int64_t{1} << 31) - 1) / kProbMaxCluster ||
      ld_logits >= (int64_t{1} << 31) || ld_probs >= (int64_t{1} << 31))
    return RLK_ERR_UNSUPPORTED_SHAPE;
  if (R == 0) return RLK_OK;
  if (!logits || !probs || !workspace) return RLK_ERR_INVALID_ARG;
  if (!al(logits, logits_type == RLK_TYPE_F32 ? 4 : 2) || !al(probs, probs_type == RLK_TYPE_F32 ? 4 : 2) ||
      !al(row_temperature, 4) || !al(workspace, 256))
    return RLK_ERR_MISALIGNED;
  // in place, a row's CTAs write where others still read unless type and stride are equal
  if (probs == logits && (probs_type != logits_type || (R > 1 && ld_probs != ld_logits)))
    return RLK_ERR_INVALID_ARG;
  if (workspace_bytes < kSampHeader) return RLK_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  rlk_status s = current_device_supported(&sms);
  if (s != RLK_OK) return s;
  ProbArgs a;
  a.x = logits;
  a.p = probs;
  a.row_tau = row_temperature;
  a.ldx = ld_logits;
  a.ldp = ld_probs;
  a.R = R;
  a.V = static_cast<int>(V);
  a.tau = temperature;
  a.err = static_cast<unsigned*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (logits_type == RLK_TYPE_F32)
    return probs_type == RLK_TYPE_F32 ? launch_probs<float, float>(a, st)
                                      : launch_probs<float, __nv_bfloat16>(a, st);
  return probs_type == RLK_TYPE_F32 ? launch_probs<__nv_bfloat16, float>(a, st)
                                    : launch_probs<__nv_bfloat16, __nv_bfloat16>(a, st);
}

extern "C" rlk_status rlk_draft_verify(const void* target_probs, int64_t target_stride_b,
                                       int64_t target_stride_k, const void* draft_probs,
                                       int64_t draft_stride_b, int64_t draft_stride_k,
                                       int probs_type, const int64_t* draft_tokens,
                                       const float* u_accept, const float* u_sample,
                                       const int64_t* draft_lens, int64_t B, int64_t K, int64_t V,
                                       int64_t* tokens, int64_t* num_accepted, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (B < 0 || K < 0 || V <= 0) return RLK_ERR_INVALID_ARG;
  if (probs_type != RLK_TYPE_BF16 && probs_type != RLK_TYPE_F32) return RLK_ERR_INVALID_ARG;
  if (target_stride_b < 0 || target_stride_k < 0 || draft_stride_b < 0 || draft_stride_k < 0)
    return RLK_ERR_INVALID_ARG;
  if (V >= (int64_t{1} << 31) || K >= (int64_t{1} << 20) ||
      B > ((int64_t{1} << 31) - 1) / kVerMaxCluster)
    return RLK_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return RLK_OK;
  if (!target_probs || !u_sample || !tokens || !num_accepted || !workspace ||
      (K > 0 && (!draft_tokens || !u_accept)))
    return RLK_ERR_INVALID_ARG;
  const uintptr_t es = probs_type == RLK_TYPE_F32 ? 4 : 2;
  if (!al(target_probs, es) || !al(draft_probs, es) || !al(draft_tokens, 8) || !al(u_accept, 4) ||
      !al(u_sample, 4) || !al(draft_lens, 8) || !al(tokens, 8) || !al(num_accepted, 8) ||
      !al(workspace, 256))
    return RLK_ERR_MISALIGNED;
  if (workspace_bytes < kSampHeader) return RLK_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  rlk_status s = current_device_supported(&sms);
  if (s != RLK_OK) return s;
  VerifyArgs a;
  a.p = target_probs;
  a.q = K > 0 ? draft_probs : nullptr;
  a.p_sb = target_stride_b;
  a.p_sk = target_stride_k;
  a.q_sb = draft_stride_b;
  a.q_sk = draft_stride_k;
  a.drafts = draft_tokens;
  a.ua = u_accept;
  a.us = u_sample;
  a.lens = draft_lens;
  a.K = K;
  a.V = static_cast<int>(V);
  a.tokens = tokens;
  a.accepted = num_accepted;
  a.err = static_cast<unsigned*>(workspace);
  a.seg = kVerPiece;
  while ((V - 1) / a.seg >= kVerMaxSegs) a.seg *= 2;
  a.nseg = static_cast<int>((V - 1) / a.seg + 1);
  // as many CTAs as run at once (two per SM), each with a segment per warp at least
  int C = 1;
  while (C < kVerMaxCluster && B * C * 2 <= 2 * sms && a.nseg >= 2 * C * kVerWarps) C *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return probs_type == RLK_TYPE_F32
             ? launch_clusters(verify_kernel<float>, a, B, C, kVerThreads, st)
             : launch_clusters(verify_kernel<__nv_bfloat16>, a, B, C, kVerThreads, st);
}
