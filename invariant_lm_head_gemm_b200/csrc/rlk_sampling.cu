// rlk_sampling.cu -- what a rollout does with a row of logits: probabilities
// at the row's temperature, and the verification of drafted tokens against the
// target's probabilities from given random numbers.
//
// Both are bound by the one pass over the rows they read (and, for the
// probabilities, write).  A row is the work of one thread-block cluster whose
// size follows from V alone: every sum then has an order that depends on V
// only, so a row's results do not depend on how many rows there are or where
// it sits.  Lanes take consecutive elements one by one, which coalesces at any
// row alignment (an odd V puts every row at another offset) and keeps the
// element-to-thread map, and with it the order of the sums, the same for all
// rows.
#include <climits>
#include <cmath>
#include <cstdint>

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
// Each thread keeps its elements in registers (kN of them, all loads in flight
// at once), so a row is read once.  Each warp takes its own maximum m_w and its
// sum relative to m_w; the pairs (m_w, s_w) of all warps of the cluster meet in
// every CTA's shared memory, one cluster barrier later every warp folds them in
// the same order, and the numerators already in registers need one more
// factor, 2^((m_w - m) k) / S.  Rows beyond the registers of eight CTAs
// (kResident = false) are read twice, the numerators formed again.
constexpr int kProbMaxWarps = 16;
constexpr int kProbMaxCluster = 8;

struct ProbArgs {
  const void* x;
  void* p;
  const float* row_tau;
  int64_t ldx, ldp;
  int V;
  int slice;  // entries per CTA of the cluster
  float tau;
  unsigned* err;
};

template <typename TIn, typename TOut, int kThreads, int kN, int kBlocks, bool kResident>
__global__ void __launch_bounds__(kThreads, kBlocks) probs_kernel(const ProbArgs P) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kStep = kN * kThreads;
  __shared__ uint2 pairs[kProbMaxCluster * kProbMaxWarps];
  uint32_t C, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  cluster_started();
  const int row = blockIdx.x / C;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lo = static_cast<int>(min(static_cast<int64_t>(rank) * P.slice, static_cast<int64_t>(P.V)));
  const int n = min(P.slice, P.V - lo);  // this CTA's entries
  const int t = threadIdx.x;
  const TIn* x = static_cast<const TIn*>(P.x) + row * P.ldx + lo;
  TOut* p = static_cast<TOut*>(P.p) + row * P.ldp + lo;

  float v[kN];
  auto load = [&](int b) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = t < n - b - j * kThreads ? to_f32(x[b + t + j * kThreads]) : -INFINITY;
  };
  float m = -INFINITY;
  const float tau = P.row_tau ? P.row_tau[row] : P.tau;
  const float k = kSampLog2e / tau;
  const bool greedy = tau == 0.f;
  for (int b = 0; b < (kResident ? 1 : n); b += kStep) {
    load(b);
#pragma unroll
    for (int j = 0; j < kN; ++j) m = fmaxf(m, v[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  const float mref = m == -INFINITY ? 0.f : m;  // -inf - -inf would be NaN

  if (greedy) {
    // this warp's first maximum; a NaN travels as the maximum
    int first = INT_MAX;
    bool nan = false;
    for (int b = 0; b < (kResident ? 1 : n); b += kStep) {
      if (!kResident) load(b);
#pragma unroll
      for (int j = kN - 1; j >= 0; --j) {
        const int i = b + t + j * kThreads;
        nan |= v[j] != v[j];
        if (i < n && v[j] == m) first = min(first, lo + i);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first = min(first, __shfl_xor_sync(kFull, first, o));
    if (__any_sync(kFull, nan)) m = NAN;
    cluster_all_started();
    if (lane < C)
      st_cluster_v2(mapa_shared(smem_u32(&pairs[rank * kWarps + warp]), lane), __float_as_uint(m),
                    static_cast<uint32_t>(first));
    cluster_sync();
    float gm = -INFINITY;
    bool bad = false;
    for (int i = lane; i < static_cast<int>(C) * kWarps; i += 32) {
      const float mi = __uint_as_float(pairs[i].x);
      gm = fmaxf(gm, mi);
      bad |= mi != mi;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(kFull, gm, o));
    bad = __any_sync(kFull, bad);
    int at = INT_MAX;
    for (int i = lane; i < static_cast<int>(C) * kWarps; i += 32)
      if (__uint_as_float(pairs[i].x) == gm) at = min(at, static_cast<int>(pairs[i].y));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) at = min(at, __shfl_xor_sync(kFull, at, o));
    const bool empty = gm == -INFINITY;
    for (int i = t; i < n; i += kThreads)
      store_as(p + i, bad ? NAN : (lo + i == at && !empty) ? 1.f : 0.f);
    if ((bad || empty) && rank == 0 && t == 0) atomicOr(P.err, RLK_DEVERR_PROBS);
    return;
  }

  // this warp's numerators and their sum, relative to its maximum
  float s = 0.f;
  for (int b = 0; b < (kResident ? 1 : n); b += kStep) {
    if (!kResident) load(b);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      v[j] = ex2_approx((v[j] - mref) * k);
      s += v[j];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
  cluster_all_started();
  if (lane < C)
    st_cluster_v2(mapa_shared(smem_u32(&pairs[rank * kWarps + warp]), lane), __float_as_uint(m),
                  __float_as_uint(s));
  cluster_sync();
  float gm = -INFINITY, S = 0.f;
  for (int i = lane; i < static_cast<int>(C) * kWarps; i += 32)
    gm = fmaxf(gm, __uint_as_float(pairs[i].x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(kFull, gm, o));
  const float gref = gm == -INFINITY ? 0.f : gm;
  for (int i = lane; i < static_cast<int>(C) * kWarps; i += 32)
    S += __uint_as_float(pairs[i].y) * ex2_approx((__uint_as_float(pairs[i].x) - gref) * k);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(kFull, S, o);
  // nothing left by the mask: all zeros; a NaN or +inf logit, or a temperature
  // that is not a positive finite number: all NaN
  const bool usable = tau > 0.f && k > 0.f && k < INFINITY && S == S;
  const bool empty = usable && gm == -INFINITY;
  float f = ex2_approx((mref - gref) * k) / S;
  if (m == -INFINITY || empty) f = 0.f;
  if (!usable) f = NAN;
  for (int b = 0; b < (kResident ? 1 : n); b += kStep) {
    if (!kResident) {
      load(b);
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = ex2_approx((v[j] - mref) * k);
    }
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if (t < n - b - j * kThreads) store_as(p + b + t + j * kThreads, v[j] * f);
  }
  if ((!usable || empty) && rank == 0 && t == 0) atomicOr(P.err, RLK_DEVERR_PROBS);
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
// The vocabulary is cut into C * kVerWarps contiguous segments, one per warp
// of the cluster.  Pass 1 sums every segment; the totals meet in every CTA's
// shared memory; every warp finds the segment that the threshold falls in, and
// the warp that owns it walks it once more (from L2) in order.
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerMaxCluster = 8;
constexpr int kVerUnroll = 10;
constexpr int kVerPiece = 1024;  // elements walked at a time: 32 consecutive ones per lane

struct VerifyArgs {
  const void* p;
  const void* q;  // null: the draft has probability one at its own token
  int64_t p_sb, p_sk, q_sb, q_sk;
  const int64_t* drafts;
  const float* ua;
  const float* us;
  const int64_t* lens;
  int64_t K, V;
  int seg;  // entries per warp, a multiple of 32
  int64_t* tokens;
  int64_t* accepted;
  unsigned* err;
};

__device__ __forceinline__ double residual(float p, float q) {
  const double d = static_cast<double>(p) - static_cast<double>(q);
  return d < 0. ? 0. : d;  // a NaN stays one
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const VerifyArgs P) {
  __shared__ double totals[2][kVerMaxCluster * kVerWarps];
  __shared__ double walk[32 * 33];
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
  int64_t len = P.lens ? P.lens[b] : P.K;
  len = len < 0 ? 0 : len > P.K ? P.K : len;

  if (warp == 0) {  // the acceptance tests, 32 drafts at a time
    int n = static_cast<int>(len);
    bool outside = false;
    for (int64_t k0 = 0; k0 < len; k0 += 32) {
      const int64_t k = k0 + lane;
      bool ok = true;
      if (k < len) {
        const int64_t d = drafts[k];
        const double u = P.ua[b * P.K + k];
        ok = d >= 0 && d < P.V;
        outside |= !ok;
        if (ok) {
          const double pd = to_f32(pb[k * P.p_sk + d]);
          const double qd = P.q ? static_cast<double>(to_f32(qb[k * P.q_sk + d])) : 1.;
          ok = u * qd < pd;
        }
      }
      const uint32_t no = __ballot_sync(kFull, !ok);
      if (no && n == static_cast<int>(len)) n = static_cast<int>(k0) + __ffs(no) - 1;
    }
    if (__any_sync(kFull, outside) && lane == 0 && rank == 0) atomicOr(P.err, RLK_DEVERR_TARGET);
    if (lane == 0) s_n = n;
    if (rank == 0) {
      for (int64_t k = lane; k <= P.K; k += 32)
        if (k != n) P.tokens[b * (P.K + 1) + k] = k < n ? drafts[k] : -1;
      if (lane == 0) P.accepted[b] = n;
    }
  }
  __syncthreads();
  const int n = s_n;
  const T* p = pb + n * P.p_sk;
  const T* q = n < len && P.q ? qb + n * P.q_sk : nullptr;
  // where q is one; a draft outside [0, V) is nowhere
  const int64_t drafted = n < len && !P.q ? drafts[n] : -1;
  const int hot = drafted >= 0 && drafted < P.V ? static_cast<int>(drafted) : -1;

  // this warp's segment
  const int nseg = static_cast<int>(C) * kVerWarps;
  const int my = static_cast<int>(rank) * kVerWarps + warp;
  const int V = static_cast<int>(P.V);
  const int lo = static_cast<int>(min(static_cast<int64_t>(my) * P.seg, P.V));
  const int hi = lo + min(P.seg, V - lo);

  for (int attempt = 0;; ++attempt) {
    const bool sub = attempt == 0;  // the second time p alone
    auto value = [&](int i) -> double {
      const float qv = sub ? (q ? to_f32(q[i]) : i == hot ? 1.f : 0.f) : 0.f;
      return residual(to_f32(p[i]), qv);
    };
    // one round trip for every 2 kVerUnroll elements of a lane: the loads of a
    // round do not wait for anything but the row's number
    double acc = 0.;
    if (sub && q) {
      for (int i = lo + lane; i < hi; i += 32 * kVerUnroll) {
        float pv[kVerUnroll], qv[kVerUnroll];
#pragma unroll
        for (int j = 0; j < kVerUnroll; ++j) {
          const bool in = i < hi - 32 * j;
          pv[j] = in ? to_f32(p[i + 32 * j]) : 0.f;
          qv[j] = in ? to_f32(q[i + 32 * j]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kVerUnroll; ++j) acc += residual(pv[j], qv[j]);
      }
    } else {
      const int h = sub ? hot : -1;
      for (int i = lo + lane; i < hi; i += 32 * 2 * kVerUnroll) {
        float pv[2 * kVerUnroll];
#pragma unroll
        for (int j = 0; j < 2 * kVerUnroll; ++j) pv[j] = i < hi - 32 * j ? to_f32(p[i + 32 * j]) : 0.f;
#pragma unroll
        for (int j = 0; j < 2 * kVerUnroll; ++j)
          acc += residual(pv[j], i + 32 * j == h ? 1.f : 0.f);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
    if (sub) cluster_all_started();
    if (lane < C) {
      const uint32_t to = mapa_shared(smem_u32(&totals[attempt][my]), lane);
      st_cluster_v2(to, static_cast<uint32_t>(__double2loint(acc)),
                    static_cast<uint32_t>(__double2hiint(acc)));
    }
    cluster_sync();

    // every warp: the running sums over the segments, four of them per lane
    constexpr int kPer = kVerMaxCluster * kVerWarps / 32;
    double t[kPer], own = 0.;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      t[j] = lane * kPer + j < nseg ? totals[attempt][lane * kPer + j] : 0.;
      own += t[j];
    }
    double incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    const double S = __shfl_sync(kFull, incl, 31);
    double excl = __shfl_up_sync(kFull, incl, 1);
    if (lane == 0) excl = 0.;
    if (S == 0. && attempt == 0 && n < len) continue;  // p <= q everywhere: take p
    const bool good = S > 0. && S < static_cast<double>(INFINITY);
    if (!good) {
      if (rank == 0 && threadIdx.x == 0) {
        P.tokens[b * (P.K + 1) + n] = -1;
        atomicOr(P.err, RLK_DEVERR_PROBS);
      }
      return;  // every warp of the cluster alike
    }
    const double c = static_cast<double>(P.us[b]) * S;
    int found = 0x7fffffff, last = -1;
    double before = 0., run = excl;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (t[j] > 0. && run + t[j] > c && found == 0x7fffffff) {
        found = lane * kPer + j;
        before = run;
      }
      run += t[j];
      if (t[j] > 0.) last = lane * kPer + j;
    }
    const uint32_t who = __ballot_sync(kFull, found != 0x7fffffff);
    // us >= 1 (or NaN): the last token of positive residual
    const bool open = who == 0 || !(P.us[b] < 1.f);
    if (!open) {
      found = __shfl_sync(kFull, found, __ffs(who) - 1);
      before = __shfl_sync(kFull, before, __ffs(who) - 1);
    } else {
      const uint32_t some = __ballot_sync(kFull, last >= 0);
      found = __shfl_sync(kFull, last, 31 - __clz(some));
    }
    if (found != my) return;

    // the owner walks its segment in order
    int fallback = -1, token = -1;
    for (int i0 = lo; i0 < hi && token < 0; i0 += kVerPiece) {
      __syncwarp();
#pragma unroll 8
      for (int j = 0; j < 32; ++j) {
        const int i = i0 + j * 32 + lane;
        walk[j * 33 + lane] = j * 32 + lane < hi - i0 ? value(i) : 0.;
      }
      __syncwarp();
      const double* w = walk + lane * 33;
      double sum = 0.;
      int lastpos = -1;
#pragma unroll 8
      for (int j = 0; j < 32; ++j) {
        sum += w[j];
        if (w[j] > 0.) lastpos = j;
      }
      double in = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(kFull, in, o);
        if (lane >= o) in += up;
      }
      double ex = __shfl_up_sync(kFull, in, 1);
      if (lane == 0) ex = 0.;
      const uint32_t cross = __ballot_sync(kFull, !open && lastpos >= 0 && before + in > c);
      const uint32_t pos = __ballot_sync(kFull, lastpos >= 0);
      if (cross) {
        const int l = __ffs(cross) - 1;
        int at = lastpos;  // rounding may leave the walk a hair below the sum
        if (lane == l) {
          double r = before + ex;
          for (int j = 0; j < 32; ++j) {
            r += w[j];
            if (w[j] > 0. && r > c) {
              at = j;
              break;
            }
          }
        }
        token = i0 + l * 32 + __shfl_sync(kFull, at, l);
      } else if (pos) {
        const int l = 31 - __clz(pos);
        fallback = i0 + l * 32 + __shfl_sync(kFull, lastpos, l);
      }
      before += __shfl_sync(kFull, in, 31);
    }
    if (lane == 0) P.tokens[b * (P.K + 1) + n] = token >= 0 ? token : fallback;
    return;
  }
}

bool al(const void* p, uintptr_t m) { return reinterpret_cast<uintptr_t>(p) % m == 0; }

template <typename Args>
rlk_status launch_clusters(void (*kern)(Args), const Args& a, int64_t groups, int C, int threads,
                           cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
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

template <typename TIn, typename TOut, int kThreads, int kN, int kBlocks, bool kResident>
rlk_status launch_probs_as(ProbArgs a, int64_t R, int C, cudaStream_t st) {
  a.slice = (a.V - 1) / C / 32 * 32 + 32;  // V / C rounded up to whole warps
  return launch_clusters(probs_kernel<TIn, TOut, kThreads, kN, kBlocks, kResident>, a, R, C,
                         kThreads, st);
}

// The register plan of a V-entry row: 16 entries per thread on the smallest
// cluster that holds it (several small CTAs share an SM, so that one's loads run
// beside another's stores), more per thread where eight CTAs do not.
template <typename TIn, typename TOut>
rlk_status launch_probs(const ProbArgs& a, int64_t R, cudaStream_t st) {
  const int V = a.V;
  if (V <= 2048) return launch_probs_as<TIn, TOut, 256, 8, 4, true>(a, R, 1, st);
  for (int C = 1; C <= kProbMaxCluster; C *= 2)
    if (V <= C * 512 * 16) return launch_probs_as<TIn, TOut, 512, 16, 3, true>(a, R, C, st);
  if (V <= 8 * 512 * 24) return launch_probs_as<TIn, TOut, 512, 24, 2, true>(a, R, 8, st);
  if (V <= 8 * 512 * 40) return launch_probs_as<TIn, TOut, 512, 40, 2, true>(a, R, 8, st);
  return launch_probs_as<TIn, TOut, 512, 16, 3, false>(a, R, 8, st);
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
  a.V = static_cast<int>(V);
  a.tau = temperature;
  a.err = static_cast<unsigned*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (logits_type == RLK_TYPE_F32)
    return probs_type == RLK_TYPE_F32 ? launch_probs<float, float>(a, R, st)
                                      : launch_probs<float, __nv_bfloat16>(a, R, st);
  return probs_type == RLK_TYPE_F32 ? launch_probs<__nv_bfloat16, float>(a, R, st)
                                    : launch_probs<__nv_bfloat16, __nv_bfloat16>(a, R, st);
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
  a.V = V;
  a.tokens = tokens;
  a.accepted = num_accepted;
  a.err = static_cast<unsigned*>(workspace);
  const int C = V <= 4096 ? 1 : V <= 16384 ? 2 : V <= 65536 ? 4 : 8;
  a.seg = static_cast<int>((V - 1) / (C * kVerWarps) / 32 * 32 + 32);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return probs_type == RLK_TYPE_F32
             ? launch_clusters(verify_kernel<float>, a, B, C, kVerThreads, st)
             : launch_clusters(verify_kernel<__nv_bfloat16>, a, B, C, kVerThreads, st);
}
