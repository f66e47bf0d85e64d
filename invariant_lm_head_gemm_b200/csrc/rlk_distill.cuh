// rlk_distill.cuh -- the parts of distillation from a teacher's top logits that
// the linear-logp kernels do not have: the teacher's weights, sorted so that an
// epilogue walking the vocabulary meets them in order; the epilogue pieces that
// pick up a student logit, or subtract a weight, where a tile holds a teacher's
// id; and the loss.
//
//   z = hidden . W^T / tau, lse = log sum_v e^z, p = e^(z - lse)
//   a_k = g_k / tau_T, q_k = e^(a_k - L), L = log sum_k e^a_k or the teacher's own lse
//   loss = sum_k q_k (log q_k - z[id_k] + lse)
//   dx[v] = dloss (Q p[v] - sum_k q_k [v = id_k]) / tau,   Q = sum_k q_k
//
// The logits come from the same tiles, in the same epilogue, as the lse: a row's
// K logits cost one comparison per chunk and one select per hit (epilogue work
// that hides under the tile's MMAs), where gathering them by K dot products per
// row would read K rows of W for every row of hidden.  Measured at T = 2047, H = 4096,
// V = 32768: 390 us with 64 slots per row, 395 with none used (power-capped, one
// process), tensor pipe 94% active; forward and backward at T = 5980, H = 4096,
// V = 151936, K = 64: 23.4 ms, 1275 TFLOP/s of the 8 T H V that recompute makes it,
// bound as the linear-logp kernels are.  Scoring 16 rows: 198 us, W's 1.25 GB at 0.96
// of the measured copy rate.
//
// dX is rounded to bf16 for the two products, as in the linear-logp backward: the
// tensor cores' 16-bit operands.  Gradients are off by about 1.7e-3 of their norm
// before their own rounding, 2.4e-3 after it (an fp32 product rounded once: 1.7e-3);
// carrying dX in two bf16 terms would add both products once more, half of the
// backward's time.
#pragma once

#include <cstdint>

#include "rlk_gemm.cuh"

namespace rlk {

// One warp per row: the used slots sorted by (id, slot), their log weights, the
// table of where every 2^shift columns' slots begin, Q and the count.  A rank
// sort: at most K^2 / 32 comparisons per lane, from shared memory, beside the
// T x H x V product it prepares.  Sums run over the sorted slots, so a row's
// results do not depend on the order in which its slots are given.  Without the
// teacher's own lse, log q = (g - max g) / tau - log sum e^((g - max g) / tau): the
// lse itself, max g / tau + log sum, would round to the size of the logits (half
// a step at 65536 is 4e-3), and that error would scale all of the row's weights.  The
// kernel that reads all this is let in at once: only its epilogue has to wait.
template <typename TLogit>
__global__ void __launch_bounds__(128) distill_prep_kernel(
    const int64_t* __restrict__ ids, const TLogit* __restrict__ logits,
    const float* __restrict__ teacher_lse, int T, int K, int V, int shift, float tau,
    const DistillRows D) {
  __shared__ int key[4][kDisMaxK];
  __shared__ float val[4][kDisMaxK];
  __shared__ int skey[4][kDisMaxK];
  __shared__ float sval[4][kDisMaxK];
  grid_dependents_go();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + w;
  if (t >= T) return;  // warp-uniform; only warp-level synchronisation below
  int n = 0;
  bool bad = false;
  for (int k0 = 0; k0 < K; k0 += 32) {
    const int k = k0 + lane;
    int id = -1;
    float logit = 0.f;
    if (k < K) {
      const int64_t i = ids[static_cast<size_t>(t) * K + k];
      if (i >= 0 && i < V) {
        id = static_cast<int>(i);
        logit = static_cast<float>(logits[static_cast<size_t>(t) * K + k]);
      } else {
        bad |= i != -1;
      }
    }
    const uint32_t used = __ballot_sync(0xffffffffu, id >= 0);
    if (id >= 0) {
      const int at = n + __popc(used & ((1u << lane) - 1u));
      key[w][at] = id;
      val[w][at] = logit;
    }
    n += __popc(used);
  }
  bad = __any_sync(0xffffffffu, bad);
  __syncwarp();
  for (int i = lane; i < n; i += 32) {
    const int id = key[w][i];
    int r = 0;
    for (int j = 0; j < n; ++j) {
      const int o = key[w][j];
      r += (o < id || (o == id && j < i)) ? 1 : 0;
    }
    skey[w][r] = id;
    sval[w][r] = val[w][i];
  }
  __syncwarp();
  float m = -INFINITY;
  bool nan = false;
  for (int i = lane; i < n; i += 32) {
    m = fmaxf(m, sval[w][i]);
    nan |= sval[w][i] != sval[w][i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  nan = __any_sync(0xffffffffu, nan);
  if (m == -INFINITY && !nan) n = 0;  // every slot at -inf: no weight anywhere
  float ref = 0.f, L;  // log q = (g - ref) / tau - L
  if (teacher_lse != nullptr) {
    L = teacher_lse[t];
  } else {
    ref = m;
    float s = 0.f;
    for (int i = lane; i < n; i += 32) s += expf((sval[w][i] - ref) / tau);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    L = logf(s);
  }
  const size_t row0 = static_cast<size_t>(t) * D.ld;
  float Q = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float logq = (sval[w][i] - ref) / tau - L;
    Q += dis_weight(logq);
    D.ids[row0 + i] = skey[w][i];
    D.logq[row0 + i] = logq;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) Q += __shfl_xor_sync(0xffffffffu, Q, o);
  if (lane == 0) {
    D.sum[t] = Q;
    D.count[t] = n | (bad ? kDisBad : 0);
  }
  uint2* head = D.head + static_cast<size_t>(t) * D.G;
  for (int g = lane; g < D.G; g += 32) head[g] = make_uint2(kDisEnd, 0u);
  __syncwarp();  // the columns that have slots are written after all are cleared
  for (int i = lane; i < n; i += 32) {
    const int g = skey[w][i] >> shift;
    if (i > 0 && skey[w][i - 1] >> shift == g) continue;
    int lo = i + 1, hi = n;  // the first slot of a later column
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (skey[w][mid] >> shift == g) {
        lo = mid + 1;
      } else {
        hi = mid;
      }
    }
    head[g] = make_uint2(static_cast<uint32_t>(skey[w][i]), static_cast<uint32_t>(i | lo << 16));
  }
}

// combine_kernel's merge of the splits (one warp per row, the same order, so the
// same lse), then the loss over the row's sorted slots.
__global__ void __launch_bounds__(256) distill_combine_kernel(
    const float* __restrict__ pm, const float* __restrict__ ps, const float* __restrict__ pb,
    const DistillRows D, int T, int G, float* __restrict__ loss, float* __restrict__ lse,
    uint32_t* err) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= T) return;  // warp-uniform
  Triple acc{kMaskLogit, 0.f, 0.f};
  for (int g = lane; g < G; g += 32) {
    const size_t i = static_cast<size_t>(t) * G + g;
    acc = merge_triple(acc, Triple{pm[i], ps[i], pb[i]});
  }
  acc = merge_lanes(acc);
  const float l2s = log2f(acc.s);
  const int c = D.count[t], n = c & ~kDisBad;
  const size_t row0 = static_cast<size_t>(t) * D.ld;
  float sum = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float logq = D.logq[row0 + i], q = dis_weight(logq);
    const float logp = kLn2 * ((D.y[row0 + i] - acc.m) - l2s);
    sum += q == 0.f ? 0.f : q * (logq - logp);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane != 0) return;
  lse[t] = kLn2 * (acc.m + l2s);
  loss[t] = (c & kDisBad) ? __int_as_float(0x7fc00000) : sum;
  if (c & kDisBad) atomicOr(err, kDevErrTarget);
}

// Backward recompute of a logits tile into bf16 dlogits (EpiDlogits' chunk buffer
// and store), dx = coef (Q p - sum_k q_k [v = id_k]), coef = dloss / tau.
struct EpiDistill {
  struct Params {
    DistillRows D;
    const float* lse;
    const float* dloss;
    int T;
    int V;
    int c0;            // first W row of the chunk
    int x0;            // the chunk's first column of the dX matrix
    float scale_log2;  // log2(e) / tau
    float inv_tau;
  };
  struct State {
    float A, coef, all;  // all = coef Q
    int row;
    bool valid;
  };

  __device__ static void begin_unit(const Params& p, State& st, int row) {
    st.row = row;
    st.valid = row < p.T;
    st.A = st.coef = st.all = 0.f;
    if (st.valid) {
      const float Q = p.D.sum[row];
      st.A = p.lse[row] * kLog2e;
      // a row without weight has no gradient, not even 0 times a NaN or an infinity
      st.coef = Q == 0.f ? 0.f : p.inv_tau * p.dloss[row];
      st.all = st.coef * Q;
    }
  }

  __device__ static void tile(const Params& p, State& st, uint32_t taddr, int nt,
                              const CUtensorMap* store_map, uint32_t stage, int lane,
                              int warp_row0) {
    const bool any_row = warp_row0 < p.T;
    DisCursor slots;
    slots.none();
    float logq = 0.f;  // of the cursor's slot, loaded ahead like its id
    if (st.valid) {
      slots.begin(p.D, st.row, (p.c0 + nt * kBN) >> kDisBwdShift);
      if (slots.cur < slots.end) logq = p.D.logq[slots.row0 + slots.cur];
    }
#pragma unroll 1
    for (int c = 0; c < kBN / 32; ++c) {
      uint32_t r[32];
      tmem_ld32(taddr + c * 32, r);
      const int loc0 = nt * kBN + c * 32;
      const int col0 = p.c0 + loc0;
      float dx[32];
#pragma unroll
      for (int j = 0; j < 32; ++j)
        dx[j] = ex2_approx(__uint_as_float(r[j]) * p.scale_log2 - st.A) * st.all;
      if (col0 + 32 > p.V) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (col0 + j >= p.V) dx[j] = 0.f;
      }
      while (slots.nxt < col0 + 32) {
        const int d = slots.nxt - col0;
        const float hit = st.coef * dis_weight(logq);
        slots.next(p.D);
        if (slots.cur < slots.end) logq = p.D.logq[slots.row0 + slots.cur];
#pragma unroll
        for (int j = 0; j < 32; ++j) dx[j] = (j == d) ? dx[j] - hit : dx[j];
      }
      __syncwarp();
      if (any_row) store_dx_chunk(dx, store_map, stage + (c & 1) * 2048u, lane, p.x0 + loc0, warp_row0);
    }
  }
};

}  // namespace rlk
