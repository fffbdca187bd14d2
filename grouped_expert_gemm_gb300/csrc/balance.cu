// The router's balance loss with per-expert counts, and the gradient of its
// logits (the selected gates' and the loss's in one pass).
//
// The auxiliary term over sequences q of L_q live tokens:
//   p_t = softmax(z_t)            (MOE_SCORE_SOFTMAX)
//   p_t = sigma(z_t) / sum sigma  (MOE_SCORE_SIGMOID_GROUP)
//   f_qe = E / (k L_q) n_qe,  P_qe = sum_t p_te / L_q,
//   loss = alpha / S' sum_q sum_e f_qe P_qe,   S' = sequences with L_q > 0
// (the counts are constants of the gradient), so with
//   w_e = dloss alpha / S' f_qe / L_q
//   dz_te = p_te (w_e - sum_j p_tj w_j) [(1 - sigma_te) for the sigmoid]
// and for the selected experts, with the gates g_j and their gradients,
//   softmax: dz = g (dg - <g, dg>)
//   sigmoid: dz = g (1 - sigma) (dg - <g, dg> / route_scale).
//
// Bound: HBM from about 256 experts on, instructions below.  A warp (or, up to 192 experts,
// a part of one) holds a token's row in registers, so the logits are read once per pass.
// Forward: each block owns a tile of consecutive tokens; its warps keep column sums in
// registers and the block writes one partial row of sums and counts per sequence that the
// tile meets, at slot tile + sequence (that index grows by one with every step to the next
// tile or the next sequence, so no two (tile, sequence) pairs share a slot).  A second
// launch adds a sequence's slots in order: no floating-point atomics, the same bits every
// time.  65,536 x 384: forward 26.4 us (3.9 TB/s; 22 us the tiles), backward 35.5 us
// (5.8 TB/s, 87 % of the copy rate).
#include <float.h>
#include <math.h>

#include <algorithm>

#include "smem.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kFinishE = 8;  // experts per block of the second stage
constexpr int kManyBlocks = 1000;
constexpr int kBwdThreads = 256;
constexpr int kBwdRing = 3;  // rows of a warp's ring: four blocks an SM within 227 KB
constexpr int kMaxE = 512;
constexpr int kMaxK = 16;

struct BalArgs {
  int T, E, k, S;
  int sigmoid;
  int tile;       // tokens per block
  int early;      // the grid is resident at once: dependents may launch right after the wait
  float alpha, route_scale;
  const int32_t* off;  // [S + 1], or nullptr: one sequence of all tokens
  const float* logits;
  const int32_t* ids;
  // forward
  float* part_sum;     // [slots, E]
  int32_t* part_cnt;   // [slots, E]
  int32_t* part_tok;   // [slots]
  int32_t* ticket;
  double* part_loss;   // [S, expert blocks]
  int32_t* counts;     // [S, E]
  int32_t* tokens;     // [S + 1]
  float* probs;        // [S, E]
  float* loss;
  // backward
  const float* gates;
  const float* dgates;
  const float* dloss;
  float* dlogits;
  uint32_t* dev_status;
};

// Bounds of sequence q, inside [0, T] whatever the array holds.
__device__ __forceinline__ int seq_bound(const BalArgs& a, int q) {
  if (a.off == nullptr) return q == 0 ? 0 : a.T;
  return min(max(__ldg(a.off + q), 0), a.T);
}

// Last q in [0, S) with bound(q) <= t (0 if there is none).
__device__ __forceinline__ int seq_of(const BalArgs& a, int t) {
  int lo = 0, hi = a.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_bound(a, mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void check_offsets(const BalArgs& a) {
  if (a.off == nullptr || blockIdx.x != 0) return;
  bool bad = false;
  for (int q = threadIdx.x; q <= a.S; q += blockDim.x) {
    const int v = __ldg(a.off + q);
    bad |= v < 0 || v > a.T || (q > 0 && v < __ldg(a.off + q - 1));
  }
  if (bad) report(a.dev_status, MOE_DEV_BAD_MAP);
}

// A token is held by L lanes of a warp, so that a warp works on 32 / L tokens at once
// (L < 32: up to 192 experts).  `gl` is the lane's place in its group.
// The lane's values of one row: expert VEC * (gl + L i) + j in v[VEC * i + j];
// places past E hold -inf.
template <int VEC, int N, int L>
__device__ __forceinline__ void load_row(const float* row, int E, int gl, float (&v)[VEC * N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = VEC * (gl + L * i);
    if constexpr (VEC == 4) {
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) f = __ldg(reinterpret_cast<const float4*>(row + e));
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    } else {
      v[i] = e < E ? __ldg(row + e) : -INFINITY;
    }
  }
}

// A warp's ring of rows in shared memory.  Each lane copies its own values of a row
// (asynchronously, in the load_row layout) and reads only those back, so a wait for
// its own copies is all the ordering there is.  Every row is one group of copies,
// empty past the end.
template <int VEC, int N, int L, int ROWS>
struct Ring {
  static constexpr int kRow = 32 * VEC * N;  // floats
  float* base;                               // [ROWS][kRow], this warp's
  __device__ __forceinline__ void copy(const float* row, int E, int lane, int slot, bool live) {
    if (live) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = VEC * (lane % L + L * i);
        const uint32_t dst = static_cast<uint32_t>(
            __cvta_generic_to_shared(base + slot * kRow + VEC * (lane + 32 * i)));
        if (e < E) {
          if constexpr (VEC == 4)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(row + e) : "memory");
          else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(row + e) : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Waits for all but the newest `ROWS - 1` rows.
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(ROWS - 1) : "memory");
  }
  __device__ __forceinline__ void read(int E, int lane, int slot, float (&v)[VEC * N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = VEC * (lane % L + L * i);
      const float* p = base + slot * kRow + VEC * (lane + 32 * i);
      if constexpr (VEC == 4) {
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < E) f = *reinterpret_cast<const float4*>(p);
        v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
      } else {
        v[i] = e < E ? *p : -INFINITY;
      }
    }
  }
};

// Sum over the token's lanes.
template <int L>
__device__ __forceinline__ float group_add(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// Largest value over the token's lanes (NaN operands are ignored).
template <int L>
__device__ __forceinline__ float group_max(float x) {
  if constexpr (L == 32) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
  }
}

constexpr float kLog2E = 1.44269504088896341f;
constexpr float kFoldedMax = 0x1p20f;

// The instruction errs by 2^-22; results below the normal range are 0.
__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// e^x as 2^(x log2 e): two more roundings of the argument (2^-23 |x|).
__device__ __forceinline__ float exp_of(float x) { return exp2_of(x * kLog2E); }

template <int M, int L>
__device__ __forceinline__ float row_max(const float (&v)[M]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < M; ++i) m = fmaxf(m, v[i]);
  m = group_max<L>(m);
  return m == -INFINITY ? 0.0f : m;  // a row of -inf: every term is then exp(-inf) = 0
}

// Unnormalised probabilities of a row in place of its logits, and the lane's part
// of their sum.  Softmax: e^(z - max).  Sigmoid: sigma(z), in an all-negative row
// divided by e^max so that the sum cannot underflow.  `slope` receives 1 - sigma.
// A NaN or +inf in the row makes the warp's sum NaN (+inf: inf - inf; for the
// sigmoid the maximum is checked), so the common path has no test per value.
template <int M, int L, bool SIG, bool SLOPE>
__device__ __forceinline__ float row_terms(float (&v)[M], float (&slope)[SIG && SLOPE ? M : 1]) {
  const float m = row_max<M, L>(v);
  float sum = 0.0f;
  if constexpr (!SIG) {
    // e^(z - m) as 2^(z log2 e - c): the rounding of c = m log2 e is the row's own factor
    // 2^(half an ulp of c), which the sum takes out again while it is near one: 2^(1/16) at
    // most here (from |m| of about 2^30 on it would leave the type's range).
    if (fabsf(m) < kFoldedMax) {
      const float c = m * kLog2E;
#pragma unroll
      for (int i = 0; i < M; ++i) {
        v[i] = exp2_of(fmaf(v[i], kLog2E, -c));
        sum += v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        v[i] = exp_of(v[i] - m);
        sum += v[i];
      }
    }
  } else if (m >= 0.0f) {
    if (m > FLT_MAX) sum = NAN;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      // a sigma below e^-80 adds nothing to a sum >= 1/2
      const bool masked = v[i] == -INFINITY;
      const float t = exp_of(v[i] < -80.0f ? 80.0f : -v[i]);
      const float s = masked ? 0.0f : __fdividef(1.0f, 1.0f + t);
      if constexpr (SLOPE) slope[i] = masked ? 1.0f : t * s;
      v[i] = s;
      sum += s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const float r = __fdividef(1.0f, 1.0f + exp_of(v[i]));
      if constexpr (SLOPE) slope[i] = r;
      v[i] = exp_of(v[i] - m) * r;
      sum += v[i];
    }
  }
  return sum;
}

// The row again with NaN as -inf and +inf as the largest finite value, reported.
template <int VEC, int N, int L>
__device__ __forceinline__ void reload_finite(const float* row, int E, int gl,
                                              float (&v)[VEC * N], uint32_t* dev_status) {
  load_row<VEC, N, L>(row, E, gl, v);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VEC * N; ++i) {
    if (!(v[i] <= FLT_MAX)) {
      v[i] = isnan(v[i]) ? -INFINITY : FLT_MAX;
      bad = true;
    }
  }
  if (bad) report(dev_status, MOE_DEV_NONFINITE_LOGIT);
}

// A warp keeps the next token's row in flight, in registers, while it works on the
// current one (four rows in shared memory instead, as the backward does: 65,536 x 384
// with the second stage 30.6 us against 28.5 then; the pass is bound by instructions as much
// as by HBM).
template <int VEC, int N, int L, bool SIG>
__global__ void __launch_bounds__(kBalThreads, VEC * N <= 12 ? 2 : 1)
balance_tile_kernel(const BalArgs a) {
  constexpr int M = VEC * N;
  constexpr int kTokens = 32 / L, kStep = kBalWarps * kTokens;
  constexpr int kIds = (kMaxK + L - 1) / L < 4 ? (kMaxK + L - 1) / L : 4;  // (k <= E <= 4 L)
  __shared__ float s_sum[kBalWarps][L * M];
  __shared__ int32_t s_cnt[kMaxE];
  __shared__ int32_t s_tok;
  pdl_wait_then_trigger(a.early);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane % L, g = lane / L;
  check_offsets(a);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  const int t0 = blockIdx.x * a.tile, t1 = min(a.T, t0 + a.tile);
  for (int q = seq_of(a, t0); q < a.S; ++q) {
    const int b = max(seq_bound(a, q), t0), e = min(seq_bound(a, q + 1), t1);
    if (b >= t1) break;
    if (b >= e) continue;
    for (int i = threadIdx.x; i < a.E; i += kBalThreads) s_cnt[i] = 0;
    if (threadIdx.x == 0) s_tok = 0;
    __syncthreads();
    float acc[M], next[M];
#pragma unroll
    for (int i = 0; i < M; ++i) acc[i] = 0.0f;
    int live_tokens = 0, next_id[kIds];
    auto fetch = [&](int t) {
      if (L == 32 || t < e) {
        load_row<VEC, N, L>(a.logits + static_cast<int64_t>(t) * a.E, a.E, gl, next);
      } else {
#pragma unroll
        for (int i = 0; i < M; ++i) next[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < kIds; ++i)
        next_id[i] = gl + L * i < a.k && (L == 32 || t < e)
                         ? __ldg(a.ids + static_cast<int64_t>(t) * a.k + gl + L * i)
                         : MOE_ROUTE_MASKED;
    };
    const int first = b + warp * kTokens;
    if (first < e) fetch(first + g);
    for (int tw = first; tw < e; tw += kStep) {
      float v[M], none[1];
      int id[kIds];
#pragma unroll
      for (int i = 0; i < M; ++i) v[i] = next[i];
#pragma unroll
      for (int i = 0; i < kIds; ++i) id[i] = next_id[i];
      if (tw + kStep < e) fetch(tw + kStep + g);
      const bool live = __shfl_sync(0xFFFFFFFFu, id[0], lane - gl) != MOE_ROUTE_MASKED;  // no padding
      if (L == 32 ? !live : !__any_sync(0xFFFFFFFFu, live)) continue;
      float sum = group_add<L>(row_terms<M, L, SIG, false>(v, none));
      if (L == 32 ? isnan(sum) : __any_sync(0xFFFFFFFFu, live && isnan(sum))) {
        const int t = min(tw + g, e - 1);
        reload_finite<VEC, N, L>(a.logits + static_cast<int64_t>(t) * a.E, a.E, gl, v,
                                 live ? a.dev_status : nullptr);
        sum = group_add<L>(row_terms<M, L, SIG, false>(v, none));
      }
      const float inv = live && sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int i = 0; i < M; ++i) {  // (a padding token's terms may be NaN)
        if constexpr (L == 32) acc[i] += v[i] * inv;
        else acc[i] += inv != 0.0f ? v[i] * inv : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kIds; ++i) {
        if (live && gl + L * i < a.k) {
          if (id[i] >= 0 && id[i] < a.E) atomicAdd(&s_cnt[id[i]], 1);
          else if (id[i] != MOE_ROUTE_MASKED) report(a.dev_status, MOE_DEV_BAD_EXPERT_ID);
        }
      }
      live_tokens += live;
    }
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {  // the warp's tokens together
      live_tokens += __shfl_xor_sync(0xFFFFFFFFu, live_tokens, o);
#pragma unroll
      for (int i = 0; i < M; ++i) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
    }
    if (g == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s_sum[warp][VEC * (gl + L * i) + j] = acc[VEC * i + j];
    }
    if (lane == 0) atomicAdd(&s_tok, live_tokens);
    __syncthreads();
    const int64_t out = static_cast<int64_t>(blockIdx.x) + q;
    for (int i = threadIdx.x; i < a.E; i += kBalThreads) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) s += s_sum[w][i];
      a.part_sum[out * a.E + i] = s;
      a.part_cnt[out * a.E + i] = s_cnt[i];
    }
    if (threadIdx.x == 0) a.part_tok[out] = s_tok;
    __syncthreads();
  }
  if (!a.early) pdl_trigger();
}

// The block that finished last: the loss from all terms, in an order fixed by their number.
__device__ __forceinline__ void add_terms(const BalArgs& a, int64_t n_terms, double* s_loss,
                                          int32_t* s_tok) {
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  __threadfence();
  double part = 0.0;
  int used = 0;
  for (int64_t i = threadIdx.x; i < n_terms; i += kBalThreads) part += __ldcg(a.part_loss + i);
  for (int i = threadIdx.x; i < a.S; i += kBalThreads) used += __ldcg(a.tokens + i) > 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
  used = __reduce_add_sync(0xFFFFFFFFu, used);
  if (lane == 0) {
    s_loss[g] = part;
    s_tok[g] = used;
  }
  __syncthreads();
  if (g == 0) {
    part = lane < kBalWarps ? s_loss[lane] : 0.0;
    used = __reduce_add_sync(0xFFFFFFFFu, lane < kBalWarps ? s_tok[lane] : 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
    if (lane == 0) {
      a.tokens[a.S] = used;
      *a.loss = used > 0 ? static_cast<float>(a.alpha * part / used) : 0.0f;
    }
  }
}

// One block per (8 experts -- a sector of each slot --, sequence): the sequence's slots
// in order (64 interleaved groups, then 4 runs of 16 groups, then the runs).  The
// block that finishes last adds the loss terms, in an order fixed by their number.
__global__ void __launch_bounds__(kBalThreads)
balance_finish_kernel(const BalArgs a) {
  constexpr int kGroups = kBalThreads / kFinishE;
  __shared__ float s_sum[kGroups][kFinishE];
  __shared__ int32_t s_cnt[kGroups][kFinishE];
  __shared__ int32_t s_tok[kBalWarps];
  __shared__ double s_loss[kBalWarps];
  __shared__ bool last;
  pdl_wait_then_trigger(a.early);
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int eb = gridDim.x, q = blockIdx.y;
  const int b = seq_bound(a, q), end = seq_bound(a, q + 1);
  float sum = 0.0f;
  int cnt = 0, tok = 0;
  {
    const int e = blockIdx.x * kFinishE + threadIdx.x % kFinishE, group = threadIdx.x / kFinishE;
    if (b < end) {
      const int64_t first = static_cast<int64_t>(b / a.tile) + q;
      const int n = (end - 1) / a.tile - b / a.tile + 1;
      if (e < a.E) {
#pragma unroll 5
        for (int i = group; i < n; i += kGroups) {
          sum += a.part_sum[(first + i) * a.E + e];
          cnt += a.part_cnt[(first + i) * a.E + e];
        }
      }
      for (int i = threadIdx.x; i < n; i += kBalThreads) tok += a.part_tok[first + i];
    }
    s_sum[group][threadIdx.x % kFinishE] = sum;
    s_cnt[group][threadIdx.x % kFinishE] = cnt;
  }
  tok = __reduce_add_sync(0xFFFFFFFFu, tok);
  if (lane == 0) s_tok[g] = tok;
  __syncthreads();
  if (g == 0) {
    const int col = lane % kFinishE, run = lane / kFinishE;
    const int e = blockIdx.x * kFinishE + col;
    tok = 0;
#pragma unroll
    for (int i = 0; i < kBalWarps; ++i) tok += s_tok[i];
    sum = 0.0f;
    cnt = 0;
#pragma unroll
    for (int i = 0; i < kGroups / 4; ++i) {
      sum += s_sum[run * (kGroups / 4) + i][col];
      cnt += s_cnt[run * (kGroups / 4) + i][col];
    }
#pragma unroll
    for (int o = kFinishE; o < 32; o <<= 1) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      cnt += __shfl_xor_sync(0xFFFFFFFFu, cnt, o);
    }
    const float mean = tok > 0 ? sum / static_cast<float>(tok) : 0.0f;
    double term = 0.0;
    if (run == 0 && e < a.E) {
      a.counts[static_cast<int64_t>(q) * a.E + e] = cnt;
      a.probs[static_cast<int64_t>(q) * a.E + e] = mean;
      if (tok > 0) term = static_cast<double>(cnt) * mean;
    }
#pragma unroll
    for (int o = kFinishE / 2; o > 0; o >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, o);
    if (lane == 0 && gridDim.x * gridDim.y == 1) {  // nothing to wait for
      a.tokens[0] = tok;
      a.tokens[1] = tok > 0;
      *a.loss = tok > 0 ? static_cast<float>(a.alpha * (term * a.E / (static_cast<double>(a.k) * tok)))
                        : 0.0f;
      last = false;
    } else if (lane == 0) {
      if (blockIdx.x == 0) a.tokens[q] = tok;
      a.part_loss[static_cast<int64_t>(q) * eb + blockIdx.x] =
          tok > 0 ? term * a.E / (static_cast<double>(a.k) * tok) : 0.0;
      __threadfence();
      last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (last) add_terms(a, static_cast<int64_t>(a.S) * eb, s_loss, s_tok);
  if (!a.early) pdl_trigger();
}

// The same for many sequences of few slots: one block a sequence, all experts side by
// side (`cols` threads, the slots interleaved over 512 / cols groups of them).
// 65,536 x 384, 512 sequences: with a block per eight experts 165 us the forward, so 35.
__global__ void __launch_bounds__(kBalThreads)
balance_finish_many_kernel(const BalArgs a, int cols) {
  __shared__ float s_sum[kBalThreads];
  __shared__ int32_t s_cnt[kBalThreads];
  __shared__ int32_t s_tok[kBalWarps];
  __shared__ double s_loss[kBalWarps];
  __shared__ bool last;
  pdl_wait_then_trigger(a.early);
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int q = blockIdx.x, e = threadIdx.x % cols, groups = kBalThreads / cols;
  const int b = seq_bound(a, q), end = seq_bound(a, q + 1);
  float sum = 0.0f;
  int cnt = 0, tok = 0;
  if (b < end) {
    const int64_t first = static_cast<int64_t>(b / a.tile) + q;
    const int n = (end - 1) / a.tile - b / a.tile + 1;
    if (e < a.E) {
#pragma unroll 4
      for (int i = threadIdx.x / cols; i < n; i += groups) {
        sum += a.part_sum[(first + i) * a.E + e];
        cnt += a.part_cnt[(first + i) * a.E + e];
      }
    }
    for (int i = threadIdx.x; i < n; i += kBalThreads) tok += a.part_tok[first + i];
  }
  s_sum[threadIdx.x] = sum;
  s_cnt[threadIdx.x] = cnt;
  tok = __reduce_add_sync(0xFFFFFFFFu, tok);
  if (lane == 0) s_tok[g] = tok;
  __syncthreads();
  tok = 0;
#pragma unroll
  for (int i = 0; i < kBalWarps; ++i) tok += s_tok[i];
  double term = 0.0;
  if (threadIdx.x < cols && e < a.E) {
    for (int i = 1; i < groups; ++i) {
      sum += s_sum[i * cols + e];
      cnt += s_cnt[i * cols + e];
    }
    const float mean = tok > 0 ? sum / static_cast<float>(tok) : 0.0f;
    a.counts[static_cast<int64_t>(q) * a.E + e] = cnt;
    a.probs[static_cast<int64_t>(q) * a.E + e] = mean;
    if (tok > 0) term = static_cast<double>(cnt) * mean;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, o);
  if (lane == 0) s_loss[g] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kBalWarps; ++i) term += s_loss[i];
    a.tokens[q] = tok;
    a.part_loss[q] = tok > 0 ? term * a.E / (static_cast<double>(a.k) * tok) : 0.0;
    __threadfence();
    last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (last) add_terms(a, a.S, s_loss, s_tok);
  if (!a.early) pdl_trigger();
}

// The rows of a warp's next tokens on their way into the warp's ring
// (65,536 x 384: 35.5 us, 87 % of HBM, against 38.6 with one row ahead in registers,
// which left the last ones spilled).  The dot product and the sum are reduced together
// before the row is normalised; the selected experts' terms reach their lanes through a
// row of shared memory that is zero between tokens.
template <int VEC, int N, int L, bool SIG>
__global__ void __launch_bounds__(kBwdThreads, VEC * N <= 12 ? 4 : 2)
route_backward_kernel(const BalArgs a) {
  constexpr int M = VEC * N;
  constexpr int kWarps = kBwdThreads / 32;
  constexpr int kTokens = 32 / L, kStep = kWarps * kTokens;
  constexpr int kIds = (kMaxK + L - 1) / L < 4 ? (kMaxK + L - 1) / L : 4;  // (k <= E <= 4 L)
  constexpr int kRows = kBwdRing;
  __shared__ __align__(16) float s_sel[kWarps][32 * M];
  extern __shared__ __align__(16) float s_ring[];  // [warps][kRows][32 M]
  pdl_wait_then_trigger(a.early);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane % L, g = lane / L;
  float* sel = s_sel[warp] + g * (L * M);  // the token's
#pragma unroll
  for (int i = 0; i < M; ++i) s_sel[warp][lane + 32 * i] = 0.0f;
  __syncwarp();
  const bool balance = a.counts != nullptr;
  float scale = 0.0f;
  if (balance) {
    const int used = __ldg(a.tokens + a.S);
    scale = used > 0 ? a.alpha / used : 0.0f;
    if (a.dloss != nullptr) scale *= __ldg(a.dloss);
    check_offsets(a);
  }
  const int t0 = blockIdx.x * a.tile, t1 = min(a.T, t0 + a.tile);
  int seq_b = 0, seq_e = 0;  // bounds of the sequence whose weights are in w
  float w[M];
#pragma unroll
  for (int i = 0; i < M; ++i) w[i] = 0.0f;
  Ring<VEC, N, L, kRows> ring = {s_ring + warp * kRows * (32 * M)};
  int slot = 0;
  auto fetch_row = [&](int t, int to) {
    ring.copy(a.logits + static_cast<int64_t>(t) * a.E, a.E, lane, to, balance && t < t1);
  };
  int next_id[kIds];
  float next_g[kIds], next_dg[kIds];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      const int64_t at = static_cast<int64_t>(t) * a.k + gl + L * i;
      const bool in = gl + L * i < a.k && (L == 32 || t < t1);
      next_id[i] = in ? __ldg(a.ids + at) : MOE_ROUTE_MASKED;
      next_g[i] = next_dg[i] = 0.0f;
      if (a.dgates != nullptr && in) {
        next_g[i] = __ldg(a.gates + at);
        next_dg[i] = __ldg(a.dgates + at);
      }
    }
  };
  const int first = t0 + warp * kTokens;
  for (int i = 0; i < kRows - 1; ++i) fetch_row(first + g + i * kStep, i);
  if (first < t1) fetch(first + g);
  for (int tw = first; tw < t1; tw += kStep) {
    const bool in = L == 32 || tw + g < t1;
    const int t = in ? tw + g : t1 - 1;
    float v[M], slope[SIG ? M : 1];
    const float* row = a.logits + static_cast<int64_t>(t) * a.E;
    int id[kIds];
    bool ok[kIds];
    float gt[kIds], dg[kIds], inner = 0.0f;
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      id[i] = next_id[i];
      ok[i] = id[i] >= 0 && id[i] < a.E;
      gt[i] = ok[i] ? next_g[i] : 0.0f;
      dg[i] = ok[i] ? next_dg[i] : 0.0f;
      inner += gt[i] * dg[i];
    }
    fetch_row(tw + g + (kRows - 1) * kStep, slot == 0 ? kRows - 1 : slot - 1);
    if (tw + kStep < t1) fetch(tw + kStep + g);
    if (balance) {
      ring.wait();
      ring.read(a.E, lane, slot, v);
    }
    if (++slot == kRows) slot = 0;
    const bool pad = __shfl_sync(0xFFFFFFFFu, id[0], lane - gl) == MOE_ROUTE_MASKED;
    if (balance && (t < seq_b || t >= seq_e)) {
      const int q = seq_of(a, t);
      seq_b = seq_bound(a, q);
      seq_e = seq_bound(a, q + 1);
      const bool inside = t >= seq_b && t < seq_e;
      const float n = static_cast<float>(__ldg(a.tokens + q));
      const float c = inside && n > 0.0f ? scale * a.E / (a.k * n) / n : 0.0f;
      if (!inside) seq_e = seq_b;  // look again at the next token
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int e = VEC * (gl + L * i) + j;
          w[VEC * i + j] =
              e < a.E ? c * __ldg(a.counts + static_cast<int64_t>(q) * a.E + e) : 0.0f;
        }
    }
    __syncwarp();
    if (balance) {
      float sum = row_terms<M, L, SIG, true>(v, slope);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < M; ++i) dot += v[i] * w[i];
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) {  // three chains side by side
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        inner += __shfl_xor_sync(0xFFFFFFFFu, inner, o);
      }
      if (L == 32 ? isnan(sum) : __any_sync(0xFFFFFFFFu, in && isnan(sum))) {
        reload_finite<VEC, N, L>(row, a.E, gl, v, pad || !in ? nullptr : a.dev_status);
        sum = group_add<L>(row_terms<M, L, SIG, true>(v, slope));
        dot = 0.0f;
#pragma unroll
        for (int i = 0; i < M; ++i) dot += v[i] * w[i];
        dot = group_add<L>(dot);
      }
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      const float shift = dot * inv * inv;
#pragma unroll
      for (int i = 0; i < M; ++i) {
        v[i] *= fmaf(w[i], inv, -shift);
        if constexpr (SIG) v[i] *= slope[i];
      }
    } else {
      inner = group_add<L>(inner);
#pragma unroll
      for (int i = 0; i < M; ++i) v[i] = 0.0f;
    }
    if (a.dgates != nullptr && (L == 32 ? !pad : __any_sync(0xFFFFFFFFu, !pad))) {
      // each slot leaves its number at its expert: one that finds another's there shares
      // the expert (ids that moe_route did not write), and the slots are then added one by
      // one in slot order
      float dz[kIds];
      bool shared_id = false;
#pragma unroll
      for (int i = 0; i < kIds; ++i) {
        ok[i] = ok[i] && !pad;
        if (!pad && !ok[i] && id[i] != MOE_ROUTE_MASKED) report(a.dev_status, MOE_DEV_BAD_EXPERT_ID);
        dz[i] = gt[i] * (dg[i] - (SIG ? inner / a.route_scale : inner));
        if (SIG && ok[i]) {
          const float z = __ldg(row + id[i]);
          dz[i] *= __fdividef(1.0f, 1.0f + exp_of(fminf(z, 80.0f)));
        }
        if (ok[i]) sel[id[i]] = __int_as_float(gl + L * i);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kIds; ++i)
        shared_id |= ok[i] && __float_as_int(sel[id[i]]) != gl + L * i;
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, shared_id)) {
#pragma unroll
        for (int i = 0; i < kIds; ++i)
          if (ok[i]) sel[id[i]] = 0.0f;
        __syncwarp();
        for (int j = 0; j < a.k; ++j) {
#pragma unroll
          for (int i = 0; i < kIds; ++i)
            if (gl + L * i == j && ok[i]) sel[id[i]] += dz[i];
          __syncwarp();
        }
      } else {
#pragma unroll
        for (int i = 0; i < kIds; ++i)
          if (ok[i]) sel[id[i]] = dz[i];
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if constexpr (VEC == 4) {
          const float4 s = *reinterpret_cast<const float4*>(sel + 4 * (gl + L * i));
          v[4 * i] += s.x; v[4 * i + 1] += s.y; v[4 * i + 2] += s.z; v[4 * i + 3] += s.w;
        } else {
          v[i] += sel[gl + L * i];
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kIds; ++i)
        if (ok[i]) sel[id[i]] = 0.0f;
      __syncwarp();
    }
    float* out = a.dlogits + static_cast<int64_t>(t) * a.E;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = VEC * (gl + L * i);
      if (e < a.E && in) {
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(out + e) =
              pad ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                  : make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        else
          out[e] = pad ? 0.0f : v[i];
      }
    }
  }
  if (!a.early) pdl_trigger();
}

// --------------------------------- host side --------------------------------

// Few tokens spread over more lanes of more blocks, at least eight lanes a token.  Forward +
// backward, us with two or four lanes / so: 8 experts, 32 tokens 7.64 / 7.56, 256: 7.83 / 7.46,
// 1,024: 8.0 / 7.4, 4,096: 8.1 / 7.7; 4 experts 8.3 / 8.2, 8.2 / 8.1, 8.5 / 8.2, 7.84 / 7.95; 16
// experts 10.4 / 9.4, 11.1 / 11.0, 10.1 / 10.1, 10.3 / 10.5.
int width(int T, int E) { return T <= 1024 ? std::max(E, 17) : E; }

// Lanes that hold a token.
int lanes(int E) { return E <= 8 ? 2 : E <= 16 ? 4 : E <= 64 ? 8 : E <= 192 ? 16 : 32; }

// Tokens per block of the forward: two blocks per SM (few slots for the second
// launch to add), at least one token per group of lanes.  The 152 SMs stand as a number,
// not asked of the device: the workspace's size and the order of the sums follow from the
// arguments alone.
int tile_tokens(int T, int E) {
  return static_cast<int>(std::max<int64_t>(ceil_div(T, 2 * 152), kBalWarps * 32 / lanes(width(T, E))));
}

// The backward has no slots: four blocks per SM.
int backward_tokens(int T, int E) {
  return static_cast<int>(std::max<int64_t>(ceil_div(T, 4 * 152), kBwdThreads / lanes(width(T, E))));
}

int64_t slots(int T, int E, int S) { return ceil_div(T, tile_tokens(T, E)) + S; }

struct Layout {
  size_t sum, cnt, tok, ticket, loss, total;
};

Layout layout(int T, int E, int S) {
  Carver c;
  Layout l;
  const int64_t n = slots(T, E, S);
  l.sum = c.take<float>(n * E);
  l.cnt = c.take<int32_t>(n * E);
  l.tok = c.take<int32_t>(n);
  l.ticket = c.take<int32_t>(1);
  l.loss = c.take<double>(static_cast<size_t>(S) * ceil_div(E, kFinishE));
  l.total = c.off;
  return l;
}

moe_status check_balance(const moe_route_params* p, int32_t n_seq, const int32_t* off) {
  if (p == nullptr || p->T < 0 || p->E <= 0 || p->k <= 0 || p->k > p->E) return MOE_ERR_INVALID_ARG;
  if (p->score_fn != MOE_SCORE_SOFTMAX && p->score_fn != MOE_SCORE_SIGMOID_GROUP)
    return MOE_ERR_INVALID_ARG;
  if (p->score_fn == MOE_SCORE_SIGMOID_GROUP && !(p->route_scale > 0.0f && p->route_scale < 1e30f))
    return MOE_ERR_INVALID_ARG;
  if (n_seq < 1 || (off == nullptr && n_seq != 1)) return MOE_ERR_INVALID_ARG;
  // (token indexes run up to a tile past T: T / 304 and a few rows, below 2^23)
  if (p->E > kMaxE || p->k > kMaxK || n_seq > 65535 || p->T > INT32_MAX - (1 << 23) ||
      static_cast<int64_t>(p->T) * p->k >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Values per lane, in 16-byte pieces where the rows allow them, and lanes per token.
// 65,536 tokens, forward + backward, with a warp a token / so: 8 experts 13.5 + 20.7 /
// 7.2 + 4.0 us, 64: 15.9 + 20.6 / 11.9 + 8.6, 128: 19.1 + 20.9 / 16.7 + 13.9, 192: 20.5 + 25.4 /
// 18.1 + 18.2; 256 with half a warp: 20.9 + 25.8 / 23.4 + 26.6; single values, 31 experts:
// 15.3 + 17.1 / 11.8 + 8.0.
template <template <int, int, int, bool> class Launch, bool SIG>
moe_status by_width(bool vec4, const BalArgs& a, unsigned grid, cudaStream_t s) {
  const int E = width(a.T, a.E);
  if (vec4) {
    if (E <= 8) return Launch<4, 1, 2, SIG>::go(a, grid, s);
    if (E <= 16) return Launch<4, 1, 4, SIG>::go(a, grid, s);
    if (E <= 32) return Launch<4, 1, 8, SIG>::go(a, grid, s);
    if (E <= 64) return Launch<4, 2, 8, SIG>::go(a, grid, s);
    if (E <= 128) return Launch<4, 2, 16, SIG>::go(a, grid, s);
    if (E <= 192) return Launch<4, 3, 16, SIG>::go(a, grid, s);
    if (E <= 256) return Launch<4, 2, 32, SIG>::go(a, grid, s);
    if (E <= 384) return Launch<4, 3, 32, SIG>::go(a, grid, s);
    return Launch<4, 4, 32, SIG>::go(a, grid, s);
  }
  if (E <= 8) return Launch<1, 4, 2, SIG>::go(a, grid, s);
  if (E <= 16) return Launch<1, 4, 4, SIG>::go(a, grid, s);
  if (E <= 32) return Launch<1, 4, 8, SIG>::go(a, grid, s);
  if (E <= 64) return Launch<1, 8, 8, SIG>::go(a, grid, s);
  if (E <= 128) return Launch<1, 8, 16, SIG>::go(a, grid, s);
  if (E <= 192) return Launch<1, 12, 16, SIG>::go(a, grid, s);
  if (E <= 256) return Launch<1, 8, 32, SIG>::go(a, grid, s);
  return Launch<1, 16, 32, SIG>::go(a, grid, s);
}

template <template <int, int, int, bool> class Launch>
moe_status by_score(bool vec4, const BalArgs& a, unsigned grid, cudaStream_t s) {
  return a.sigmoid ? by_width<Launch, true>(vec4, a, grid, s)
                   : by_width<Launch, false>(vec4, a, grid, s);
}

template <int VEC, int N, int L, bool SIG>
struct TileLaunch {
  static moe_status go(const BalArgs& a, unsigned grid, cudaStream_t s) {
    launch(balance_tile_kernel<VEC, N, L, SIG>, dim3(grid), dim3(kBalThreads), 0, s, a);
    return MOE_OK;
  }
};

template <int VEC, int N, int L, bool SIG>
struct BackwardLaunch {
  static moe_status go(const BalArgs& a, unsigned grid, cudaStream_t s) {
    constexpr int kSmem = kBwdThreads / 32 * kBwdRing * 32 * VEC * N * 4;
    static std::mutex mu;
    static bool done[64] = {};
    if (!opt_in(route_backward_kernel<VEC, N, L, SIG>, kSmem, mu, done)) return MOE_ERR_CUDA;
    launch(route_backward_kernel<VEC, N, L, SIG>, dim3(grid), dim3(kBwdThreads), kSmem, s, a);
    return MOE_OK;
  }
};

BalArgs base_args(const moe_route_params* p, int32_t n_seq, const int32_t* off,
                  const float* logits, const int32_t* ids, float alpha, uint32_t* dev_status) {
  BalArgs a = {};
  a.T = p->T;
  a.E = p->E;
  a.k = p->k;
  a.S = n_seq;
  a.sigmoid = p->score_fn == MOE_SCORE_SIGMOID_GROUP;
  a.alpha = alpha;
  a.route_scale = p->route_scale;
  a.off = off;
  a.logits = logits;
  a.ids = ids;
  a.dev_status = dev_status;
  return a;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_balance_loss_workspace_size(const moe_route_params* p, int32_t n_seq) {
  const int32_t one = 0;
  if (check_balance(p, n_seq, &one) != MOE_OK) return 0;
  return layout(p->T, p->E, n_seq).total;
}

MOE_API moe_status moe_balance_loss(const moe_route_params* p, int32_t n_seq,
                                    const int32_t* seq_offsets, const float* logits,
                                    const int32_t* topk_ids, float alpha, int32_t* counts,
                                    int32_t* seq_tokens, float* mean_probs, float* loss, void* ws,
                                    size_t ws_bytes, uint32_t* dev_status, moe_stream_t stream) {
  const moe_status st = check_balance(p, n_seq, seq_offsets);
  if (st != MOE_OK) return st;
  if (counts == nullptr || seq_tokens == nullptr || mean_probs == nullptr || loss == nullptr ||
      ws == nullptr || !(fabsf(alpha) <= FLT_MAX))
    return MOE_ERR_INVALID_ARG;
  if (p->T > 0 && (logits == nullptr || topk_ids == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned4(logits) || !aligned4(topk_ids) || !aligned4(seq_offsets) || !aligned4(counts) ||
      !aligned4(seq_tokens) || !aligned4(mean_probs) || !aligned4(loss) || !aligned16(ws))
    return MOE_ERR_UNSUPPORTED;
  const Layout l = layout(p->T, p->E, n_seq);
  if (ws_bytes < l.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  BalArgs a = base_args(p, n_seq, seq_offsets, logits, topk_ids, alpha, dev_status);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.part_sum = reinterpret_cast<float*>(w + l.sum);
  a.part_cnt = reinterpret_cast<int32_t*>(w + l.cnt);
  a.part_tok = reinterpret_cast<int32_t*>(w + l.tok);
  a.ticket = reinterpret_cast<int32_t*>(w + l.ticket);
  a.part_loss = reinterpret_cast<double*>(w + l.loss);
  a.counts = counts;
  a.tokens = seq_tokens;
  a.probs = mean_probs;
  a.loss = loss;
  cudaStream_t s = as_cuda(stream);
  a.tile = tile_tokens(p->T, p->E);
  const int64_t tiles = p->T > 0 ? ceil_div(p->T, a.tile) : 1;
  a.early = one_wave(tiles);
  const moe_status tiled =
      by_score<TileLaunch>(p->E % 4 == 0 && aligned16(logits), a, static_cast<unsigned>(tiles), s);
  if (tiled != MOE_OK) return tiled;
  // Measured, us of the forward (a block per eight experts / per sequence): 65,536 x 128, 32
  // sequences 18.9 / 19.7, 64: 22.4 / 19.5; 384 experts, 16: 30.5 / 32.2, 32: 34.6 / 29.9;
  // eight experts, 4,000: 58 / 80.
  if (p->E > 32 && ceil_div(p->E, kFinishE) * n_seq >= kManyBlocks) {
    int cols = 32;
    while (cols < p->E) cols *= 2;
    a.early = one_wave(n_seq);
    launch(balance_finish_many_kernel, dim3(static_cast<unsigned>(n_seq)), dim3(kBalThreads), 0, s, a, cols);
    return launch_status();
  }
  const dim3 grid(static_cast<unsigned>(ceil_div(p->E, kFinishE)), static_cast<unsigned>(n_seq));
  a.early = one_wave(static_cast<int64_t>(grid.x) * grid.y);
  launch(balance_finish_kernel, grid, dim3(kBalThreads), 0, s, a);
  return launch_status();
}

MOE_API moe_status moe_route_backward(const moe_route_params* p, int32_t n_seq,
                                      const int32_t* seq_offsets, const float* logits,
                                      const int32_t* topk_ids, const float* gates,
                                      const float* dgates, float alpha, const int32_t* counts,
                                      const int32_t* seq_tokens, const float* dloss,
                                      float* dlogits, uint32_t* dev_status, moe_stream_t stream) {
  const moe_status st = check_balance(p, n_seq, seq_offsets);
  if (st != MOE_OK) return st;
  if ((counts == nullptr) != (seq_tokens == nullptr)) return MOE_ERR_INVALID_ARG;
  if ((dgates == nullptr && counts == nullptr) || (dgates != nullptr && gates == nullptr) ||
      !(fabsf(alpha) <= FLT_MAX))
    return MOE_ERR_INVALID_ARG;
  if (p->T == 0) return MOE_OK;
  if (logits == nullptr || topk_ids == nullptr || dlogits == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned4(logits) || !aligned4(topk_ids) || !aligned4(seq_offsets) || !aligned4(gates) ||
      !aligned4(dgates) || !aligned4(counts) || !aligned4(seq_tokens) || !aligned4(dloss) ||
      !aligned4(dlogits))
    return MOE_ERR_UNSUPPORTED;
  BalArgs a = base_args(p, n_seq, seq_offsets, logits, topk_ids, alpha, dev_status);
  a.gates = gates;
  a.dgates = dgates;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(seq_tokens);
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.tile = backward_tokens(p->T, p->E);
  const int64_t blocks = ceil_div(p->T, a.tile);
  a.early = one_wave(blocks);
  const moe_status launched =
      by_score<BackwardLaunch>(p->E % 4 == 0 && aligned16(logits) && aligned16(dlogits), a,
                               static_cast<unsigned>(blocks), as_cuda(stream));
  if (launched != MOE_OK) return launched;
  return launch_status();
}
