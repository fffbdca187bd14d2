// The tables' gradients: out[e, m, k] = sum over e's tokens of p[t, m] q[t, k], p fp32 [T, r] (u or
// v), q bf16 (dy or x); dA and dB in one launch, the columns of one behind the other's.
//
// D^T: 128 columns of q (M, their tokens the reduction, as TMA lays them down) against the r
// columns of p (N).  A CTA takes one adapter and 128 columns, and of the adapter's tokens, cut
// into pieces of up to 64 rows of one segment, all or (in a cluster) a part; parts are added in
// order.  Bound: the bytes of q.
//   warp 0      TMA producer: [64 tokens x 128] of q (16 KB) a stage
//   warp 1      tensor memory; lane 0 issues the MMAs: four of 16 tokens for each part of p
//   warps 2..5  p into the stage, transposed and as three bf16 numbers a value (the value and what
//               each rounding left: as exact as fp32); the sums onto registers every kGroup pieces
//               (the tensor cores' own fp32 sums lose 2^-26 a step); join and stores
// Rows behind a piece's last are another segment's: zeros in p, and in q, where 0 times a NaN or
// an infinity of theirs would not be zero, written over what TMA brought.
#include "adapter.cuh"

namespace moe {
namespace adapter {
namespace {

constexpr int kThreads = 192;
constexpr int kTokens = 64;
constexpr int kCols = 128;
constexpr int kQBox = kTokens * 128;
constexpr int kQBytes = 2 * kQBox;
constexpr int kGroup = 2;

template <int RB>
struct Grads {
  static constexpr int kN = 16 * RB;
  static constexpr int kPartBytes = kN * 128;  // [kN ranks][64 tokens] bf16
  static constexpr int kStageBytes = kQBytes + 3 * kPartBytes;
  static constexpr int kStages = 3;
  static constexpr int kTmem = 2 * kN < 32 ? 32 : 2 * kN;
  // full[st], ready[st], empty[st], tfull[2], tempty[2], drain
  static constexpr int kBars = 3 * kStages + 5;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kBars * 8 + 16;
  static constexpr int kPerSm = RB == 1 ? 3 : RB == 2 ? 2 : 1;
  static constexpr int kFetch = RB <= 2 ? 2 : 1;  // pieces of p on their way
  static constexpr int kItems = kN * 8 / 128;  // (rank, eight tokens) a thread of the four warps
  static_assert(kSmem * kPerSm <= 227 * 1024, "shared memory");
  static_assert(kStages * kStageBytes >= kN * kCols * 4, "sums fit the stages");
};

// The pieces of one adapter's segments, one after the other, by a whole warp.
struct Walk {
  const Segments* s;
  int id, lane;
  int q_base = -32;
  uint32_t mask = 0;
  int b = 0, e = 0;  // rows left of the current segment
  __device__ __forceinline__ Walk(const Segments& seg, int adapter, int l) : s(&seg), id(adapter), lane(l) {}
  __device__ __forceinline__ bool segment() {
    while (true) {
      while (mask == 0) {
        q_base += 32;
        if (q_base >= s->n_seg) return false;
        const int cand = q_base + lane < s->n_seg ? __ldg(s->adapter + q_base + lane) : kNone;
        mask = __ballot_sync(0xFFFFFFFFu, cand == id);
      }
      const int q = q_base + __ffs(mask) - 1;
      mask &= mask - 1;
      seg_rows(*s, q, b, e);
      if (b < e) return true;
    }
  }
  // Steps over `n` pieces (at most those that are left).
  __device__ __forceinline__ void skip(int64_t n) {
    while (n > 0) {
      if (b >= e && !segment()) return;
      const int here = (e - b + kTokens - 1) / kTokens;
      const int k = static_cast<int>(n < here ? n : here);
      b = k == here ? e : b + k * kTokens;
      n -= k;
    }
  }
  __device__ __forceinline__ bool next(int& row, int& rows) {
    if (b >= e && !segment()) return false;
    row = b;
    rows = min(e - b, kTokens);
    b += rows;
    return true;
  }
};

template <int RB>
__global__ void __launch_bounds__(kThreads, Grads<RB>::kPerSm)
grads_kernel(const __grid_constant__ CUtensorMap map_q0, const __grid_constant__ CUtensorMap map_q1,
             const GradArgs a, int split) {
  using F = Grads<RB>;
  constexpr int kStages = F::kStages, kN = F::kN;
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stage_base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage_base + kStages * F::kStageBytes);
  volatile int* abort_flag = reinterpret_cast<int*>(bars + F::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + F::kBars) + 1;
  uint32_t* ring_end = tmem_slot + 1;  // where the producer stopped, and whether MMAs were issued
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int block = static_cast<int>(blockIdx.x) / split, blocks0 = (a.side[0].K + kCols - 1) / kCols;
  const bool second = block >= blocks0;
  const CUtensorMap* map_q = second ? &map_q1 : &map_q0;
  const int K = a.side[second].K, col0 = (second ? block - blocks0 : block) * kCols;
  const float* p = a.side[second].p;
  const int id = blockIdx.y;
  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto ready_bar = [&](int s) { return smem_u32(bars + kStages + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + 2 * kStages + s); };
  auto tfull_bar = [&](int b) { return smem_u32(bars + 3 * kStages + b); };
  auto tempty_bar = [&](int b) { return smem_u32(bars + 3 * kStages + 2 + b); };
  const uint32_t drain_bar = smem_u32(bars + 3 * kStages + 4);

  pdl_wait();
  pdl_trigger();
  if (a.check && blockIdx.x == 0 && blockIdx.y == 0) check_segments(a.seg, a.dev_status);
  // the adapter's pieces: this CTA's part of them
  int64_t count = 0;
  for (int q0 = 0; q0 < a.seg.n_seg; q0 += 32) {
    int n = 0;
    if (q0 + lane < a.seg.n_seg && __ldg(a.seg.adapter + q0 + lane) == id) {
      int b, e;
      seg_rows(a.seg, q0 + lane, b, e);
      n = e > b ? (e - b + kTokens - 1) / kTokens : 0;
    }
    count += __reduce_add_sync(kAll, n);
  }
  float* out = a.side[second].out + static_cast<int64_t>(id) * a.r * K;
  if (count == 0) {  // (the same in every CTA of a cluster)
    if (rank == 0 && !a.accumulate)
      for (int i = threadIdx.x; i < a.r * kCols; i += kThreads)
        if (col0 + i % kCols < K) out[static_cast<int64_t>(i / kCols) * K + col0 + i % kCols] = 0.0f;
    return;
  }
  const int64_t part0 = count * rank / split, part1 = count * (rank + 1) / split;
  const int pieces = static_cast<int>(part1 - part0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(ready_bar(s), 4);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) umma_alloc(smem_u32(tmem_slot), F::kTmem);
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const uint32_t tmem = *tmem_slot;

  bool ok = true;
  if (warp == 0) {
    Walk w(a.seg, id, lane);
    w.skip(part0);
    int s = 0, row, rows;
    uint32_t ph = 0;
    for (int i = 0; i < pieces && w.next(row, rows); ++i) {
      ok = __all_sync(kAll, wait_bounded(empty_bar(s), ph ^ 1u, abort_flag, a.dev_status));
      if (!ok) break;
      if (lane == 0) {
        const uint32_t st = smem_u32(stage_base + s * F::kStageBytes);
        mbar_arrive_expect_tx(full_bar(s), kQBytes);
        tma_load_2d(st, map_q, full_bar(s), col0, row);
        tma_load_2d(st + kQBox, map_q, full_bar(s), col0 + 64, row);
      }
      if (++s == kStages) { s = 0; ph ^= 1u; }
    }
    if (lane == 0) ring_end[0] = static_cast<uint32_t>(s) << 1 | ph;
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = umma_idesc_bf16(128, kN, true);
      int s = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool issued = false;
      for (int i = 0; i < pieces; ++i) {
        if (i % kGroup == 0) {
          if (!wait_bounded(tempty_bar(buf), acc_ph ^ 1u, abort_flag, a.dev_status)) { ok = false; break; }
          umma_fence_after();
        }
        if (!wait_bounded(full_bar(s), ph, abort_flag, a.dev_status) ||
            !wait_bounded(ready_bar(s), ph, abort_flag, a.dev_status)) {
          ok = false;
          break;
        }
        umma_fence_after();
        const uint32_t st = smem_u32(stage_base + s * F::kStageBytes);
#pragma unroll
        for (int h = 0; h < 3; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + buf * kN, umma_desc_mn(st + kk * 16 * 128, kQBox),
                      umma_desc(st + kQBytes + h * F::kPartBytes + kk * 32), idesc,
                      i % kGroup > 0 || h > 0 || kk > 0);
        issued = true;
        umma_commit(empty_bar(s));
        if (++s == kStages) { s = 0; ph ^= 1u; }
        if (i % kGroup == kGroup - 1 || i + 1 == pieces) {
          umma_commit(tfull_bar(buf));
          if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
        }
      }
      ring_end[1] = issued;
    }
  } else {
    const int tid = threadIdx.x - 64, quad = warp & 3;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    float acc[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) acc[i] = 0.0f;
    int buf = 0, done = 0;  // pieces whose sums have been taken
    uint32_t acc_ph = 0;
    auto take = [&]() {
      if (!__all_sync(kAll, wait_bounded(tfull_bar(buf), acc_ph, abort_flag, a.dev_status))) return false;
      umma_fence_after();
#pragma unroll
      for (int c = 0; c < kN; c += 16) {
        uint32_t v[16];
        umma_ld16(taddr + buf * kN + c, v);
        umma_ld_wait(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c + i] += __uint_as_float(v[i]);
      }
      umma_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty_bar(buf));
      if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
      done = min(done + kGroup, pieces);
      return true;
    };
    // item i of this thread: rank (tid + 128 i) % kN, eight tokens from 8 ((tid + 128 i) / kN)
    float ahead[F::kFetch][F::kItems][8];
    int live[F::kFetch];
    Walk w(a.seg, id, lane);
    w.skip(part0);
    auto fetch = [&](int f) {
      int row = 0, rows = 0;
      w.next(row, rows);
      live[f] = rows;
#pragma unroll
      for (int i = 0; i < F::kItems; ++i) {
        const int item = tid + 128 * i, m = item % kN, t0 = item / kN * 8;
#pragma unroll
        for (int t = 0; t < 8; ++t)
          ahead[f][i][t] = m < a.r && t0 + t < rows ? p[static_cast<int64_t>(row + t0 + t) * a.r + m] : 0.0f;
      }
    };
    int s = 0;
    uint32_t ph = 0;
#pragma unroll
    for (int f = 0; f < F::kFetch; ++f)
      if (f < pieces) fetch(f);
    auto stage = [&](int n, int f) {  // piece n, fetched into f
      ok = __all_sync(kAll, wait_bounded(empty_bar(s), ph ^ 1u, abort_flag, a.dev_status));
      if (!ok) return;
      uint8_t* st = stage_base + s * F::kStageBytes;
#pragma unroll
      for (int i = 0; i < F::kItems; ++i) {
        const int item = tid + 128 * i, m = item % kN, j = item / kN;
        uint8_t* dst = st + kQBytes + m * 128 + ((j ^ (m & 7)) << 4);
        float f8[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) f8[t] = ahead[f][i][t];
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          uint32_t x[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            x[t] = pack_bf16x2(f8[2 * t], f8[2 * t + 1]);
            f8[2 * t] -= __uint_as_float(x[t] << 16);
            f8[2 * t + 1] -= __uint_as_float(x[t] & 0xFFFF0000u);
          }
          *reinterpret_cast<uint4*>(dst + h * F::kPartBytes) = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      const int rows = live[f];
      if (n + F::kFetch < pieces) fetch(f);
      if (rows < kTokens) {
        ok = __all_sync(kAll, wait_bounded(full_bar(s), ph, abort_flag, a.dev_status));
        if (!ok) return;
        for (int i = tid; i < (kTokens - rows) * 16; i += 128) {
          const int t = rows + i / 16, c = i % 16;
          *reinterpret_cast<uint4*>(st + c / 8 * kQBox + t * 128 + c % 8 * 16) = make_uint4(0, 0, 0, 0);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(ready_bar(s));
      if (++s == kStages) { s = 0; ph ^= 1u; }
      // the group before the one that was just staged
      if (n % kGroup == kGroup - 1 && n >= 2 * kGroup - 1) ok = take();
    };
    for (int n = 0; n < pieces && ok; n += F::kFetch) {
#pragma unroll
      for (int f = 0; f < F::kFetch; ++f)
        if (n + f < pieces && ok) stage(n + f, f);
    }
    while (ok && done < pieces) ok = take();
    const int c = quad * 32 + lane;
    if (ok && split == 1) {
      if (col0 + c < K) {
#pragma unroll
        for (int m = 0; m < kN; ++m)
          if (m < a.r) {
            float* dst = out + static_cast<int64_t>(m) * K + col0 + c;
            *dst = a.accumulate ? *dst + acc[m] : acc[m];
          }
      }
    } else if (ok) {
      // (every MMA is done, and every copy has been used: the stages are free)
      float* mine = reinterpret_cast<float*>(stage_base) + c;
#pragma unroll
      for (int m = 0; m < kN; ++m) mine[m * kCols] = acc[m];
    }
  }
  if (split > 1) {
    cluster_sync();
    if (*abort_flag == 0)
      for (int i = rank * kThreads + threadIdx.x; i < a.r * kCols; i += split * kThreads) {
        const float v = sum_of_ranks(smem_u32(reinterpret_cast<float*>(stage_base) + i), split);
        if (col0 + i % kCols < K) {
          float* dst = out + static_cast<int64_t>(i / kCols) * K + col0 + i % kCols;
          *dst = a.accumulate ? *dst + v : v;
        }
      }
    cluster_sync();  // no CTA leaves while a partner may still read its sums
  }
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  // No role gives up behind this barrier.  Where one has, whichever it was, MMAs and copies in flight end before
  // the memory that they use is given up.
  if (*abort_flag) {
    if (threadIdx.x == 32 && ring_end[1]) {
      umma_commit(drain_bar);
      wait_drain(drain_bar, 0);
    }
    if (threadIdx.x == 0) {
      int s = static_cast<int>(ring_end[0] >> 1);
      uint32_t ph = ring_end[0] & 1u;
      for (int i = 0; i < kStages; ++i) {
        if (--s < 0) { s = kStages - 1; ph ^= 1u; }
        wait_drain(full_bar(s), ph);
      }
    }
    __syncwarp();
  }
  umma_fence_after();
  if (warp == 1) {
    __syncwarp();
    umma_dealloc(tmem, F::kTmem);
  }
}

template <int RB>
moe_status launch_grads(const GradArgs& a, cudaStream_t s) {
  using F = Grads<RB>;
  auto kern = grads_kernel<RB>;
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, F::kSmem, mu, done)) return MOE_ERR_CUDA;
  CUtensorMap mq[2] = {};
  int64_t blocks = 0;
  for (int i = 0; i < 2; ++i) {
    const GradSide& g = a.side[i];
    if (g.K > 0 && !map_2d(&mq[i], g.q, a.seg.T, g.K, g.q_stride, kTokens)) return MOE_ERR_CUDA;
    blocks += ceil_div(g.K, kCols);
  }
  // Adapters that can have tokens.  Their tokens are split until the CTAs are twice what the SMs
  // hold, two pieces a CTA at least: adapters have more and less of them (4,096 tokens x 7168, of
  // which one adapter of four has 2,345: 26 us where the CTAs just fit).
  const int64_t active = std::min(a.seg.n_adapters, a.seg.n_seg);
  const int split = pow2_at_most(
      std::min<int64_t>(2 * F::kPerSm * sm_count() / (blocks * active), a.seg.T / (2 * kTokens)), 8);
  launch_clustered(kern, dim3(static_cast<unsigned>(blocks * split), a.seg.n_adapters), kThreads, F::kSmem,
                   split, s, mq[0], mq[1], a, split);
  return launch_status();
}

}  // namespace

moe_status table_grads(const GradArgs& a, cudaStream_t s) {
  const int rb = (a.r + 15) / 16;
  if (rb == 1) return launch_grads<1>(a, s);
  if (rb == 2) return launch_grads<2>(a, s);
  if (rb <= 4) return launch_grads<4>(a, s);
  return launch_grads<8>(a, s);
}

}  // namespace adapter
}  // namespace moe
