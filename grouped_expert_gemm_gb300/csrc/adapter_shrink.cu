// u = s (x A^T) of segments of many rows.
//
// A tile is up to 128 rows of one segment (M) against the r rows of its table (N), the long side
// reduced: 128-byte boxes of x and of the table by TMA, tcgen05.mma, fp32 sums in tensor memory.
// Bound: the bytes of x.  A cluster of up to eight CTAs splits the reduction, so that the tiles
// of a batch fill the SMs and each has a deep ring of x on its way; the sums are joined through
// distributed shared memory in the order of the ranks.
//   warp 0      TMA producer: [128 rows x 64] of x (16 KB) and [r x 64] of the table a stage
//   warp 1      tensor memory; lane 0 issues four MMAs (K = 16) a stage
//   warps 2..5  every kPiece steps the sums onto registers (the tensor cores' own fp32 sums
//               lose 2^-26 a step), then the join, the scale and the stores
#include "adapter.cuh"

namespace moe {
namespace adapter {
namespace {

constexpr int kThreads = 192;
constexpr int kRows = 128;
constexpr int kXBytes = kRows * 128;
constexpr int kPieceSteps = 4;

template <int RB>
struct Long {
  static constexpr int kN = 16 * RB;
  static constexpr int kStageBytes = kXBytes + kN * 128;
  static constexpr int kStages = RB <= 2 ? 5 : RB == 4 ? 4 : 3;  // two CTAs an SM
  static constexpr int kTmem = 2 * kN < 32 ? 32 : 2 * kN;
  static constexpr int kSumPitch = kN + 4;  // floats of a row of sums
  // full[st], empty[st], tfull[2], tempty[2], drain
  static constexpr int kBars = 2 * kStages + 5;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kBars * 8 + 16;
  static_assert(kSmem <= 113 * 1024 && kTmem <= 256, "two CTAs an SM");
  static_assert(kStages * kStageBytes >= kRows * kSumPitch * 4, "sums fit the stages");
};

template <int RB>
__global__ void __launch_bounds__(kThreads, 2)
shrink_long_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_t,
                   const ShrinkArgs a, int split) {
  using F = Long<RB>;
  constexpr int kStages = F::kStages, kN = F::kN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stage_base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage_base + kStages * F::kStageBytes);
  volatile int* abort_flag = reinterpret_cast<int*>(bars + F::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + F::kBars) + 1;
  uint32_t* ring_end = tmem_slot + 1;  // where the producer stopped, and whether MMAs were issued
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int steps = (a.K + 63) / 64;
  const int k0 = rank * steps / split, k1 = (rank + 1) * steps / split;
  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + kStages + s); };
  auto tfull_bar = [&](int b) { return smem_u32(bars + 2 * kStages + b); };
  auto tempty_bar = [&](int b) { return smem_u32(bars + 2 * kStages + 2 + b); };
  const uint32_t drain_bar = smem_u32(bars + 2 * kStages + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_t)) : "memory");
  }
  if (warp == 1) umma_alloc(smem_u32(tmem_slot), F::kTmem);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) check_segments(a.seg, a.dev_status);
  const Piece p = piece_of<kThreads>(a.seg, static_cast<int>(blockIdx.x) / split, kRows);
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool live = p.rows > 0 && p.adapter >= 0;

  float acc[kN];
  bool ok = true;
  if (!live) {
    if (p.rows > 0 && rank == 0)
      for (int i = threadIdx.x; i < p.rows * a.r; i += kThreads)
        a.u[static_cast<int64_t>(p.row) * a.r + i] = 0.0f;
  } else if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      for (int k = k0; k < k1; ++k) {
        if (!wait_bounded(empty_bar(s), ph ^ 1u, abort_flag, a.dev_status)) { ok = false; break; }
        const uint32_t st = smem_u32(stage_base + s * F::kStageBytes);
        mbar_arrive_expect_tx(full_bar(s), F::kStageBytes);
        tma_load_2d(st, &map_x, full_bar(s), k * 64, p.row);
        tma_load_3d(st + kXBytes, &map_t, full_bar(s), k * 64, 0, p.adapter);
        if (++s == kStages) { s = 0; ph ^= 1u; }
      }
      ring_end[0] = static_cast<uint32_t>(s) << 1 | ph;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = umma_idesc_bf16(128, kN, false);
      int s = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool issued = false;
      for (int kp = k0; kp < k1 && ok; kp += kPieceSteps) {
        if (!wait_bounded(tempty_bar(buf), acc_ph ^ 1u, abort_flag, a.dev_status)) { ok = false; break; }
        umma_fence_after();
        for (int k = kp; k < min(kp + kPieceSteps, k1); ++k) {
          if (!wait_bounded(full_bar(s), ph, abort_flag, a.dev_status)) { ok = false; break; }
          umma_fence_after();
          const uint32_t st = smem_u32(stage_base + s * F::kStageBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + buf * kN, umma_desc(st + kk * 32), umma_desc(st + kXBytes + kk * 32), idesc,
                      k > kp || kk > 0);
          issued = true;
          umma_commit(empty_bar(s));
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        umma_commit(tfull_bar(buf));
        if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
      }
      ring_end[1] = issued;
    }
  } else {
    const int quad = warp & 3;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    int buf = 0;
    uint32_t acc_ph = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) acc[i] = 0.0f;
    for (int kp = k0; kp < k1; kp += kPieceSteps) {
      ok = __all_sync(0xFFFFFFFFu, wait_bounded(tfull_bar(buf), acc_ph, abort_flag, a.dev_status));
      if (!ok) break;
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
    }
    const int row = quad * 32 + lane;
    if (ok && split == 1) {
      if (row < p.rows) {
        const float scale = __ldg(a.scale + p.adapter);
        float* out = a.u + static_cast<int64_t>(p.row + row) * a.r;
#pragma unroll
        for (int c = 0; c < kN; c += 4)
          if (c < a.r)
            *reinterpret_cast<float4*>(out + c) =
                make_float4(scale * acc[c], scale * acc[c + 1], scale * acc[c + 2], scale * acc[c + 3]);
      }
    } else if (ok) {
      // (the last sums have been read: every MMA is done, and the stages are free)
      float* mine = reinterpret_cast<float*>(stage_base) + row * F::kSumPitch;
#pragma unroll
      for (int c = 0; c < kN; c += 4)
        *reinterpret_cast<float4*>(mine + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
    }
  }
  if (split > 1) {
    cluster_sync();
    if (live && *abort_flag == 0) {
      const float scale = __ldg(a.scale + p.adapter);
      for (int i = rank * kThreads + threadIdx.x; i < p.rows * a.r; i += split * kThreads) {
        const float v = sum_of_ranks(
            smem_u32(reinterpret_cast<float*>(stage_base) + i / a.r * F::kSumPitch + i % a.r), split);
        a.u[static_cast<int64_t>(p.row) * a.r + i] = scale * v;
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
moe_status launch_long(const ShrinkArgs& a, cudaStream_t s) {
  using F = Long<RB>;
  auto kern = shrink_long_kernel<RB>;
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, F::kSmem, mu, done)) return MOE_ERR_CUDA;
  CUtensorMap mx, mt;
  if (!map_2d(&mx, a.x, a.seg.T, a.K, a.x_stride, kRows) ||
      !map_tables(&mt, a.table, a.seg.n_adapters, a.r, a.K, F::kN))
    return MOE_ERR_CUDA;
  const int64_t tiles = ceil_div(a.seg.T, kRows) + a.seg.n_seg;
  // two CTAs an SM where half of the segments' last tiles are counted; at least four steps of 64
  // a CTA
  const int split = pow2_at_most(
      std::min<int64_t>(2 * sm_count() / (tiles - a.seg.n_seg / 2), a.K / 256), 8);
  launch_clustered(kern, dim3(static_cast<unsigned>(tiles * split)), kThreads, F::kSmem, split, s, mx, mt,
                   a, split);
  return launch_status();
}

}  // namespace

moe_status shrink_long(const ShrinkArgs& a, cudaStream_t s) {
  const int rb = (a.r + 15) / 16;
  if (rb == 1) return launch_long<1>(a, s);
  if (rb == 2) return launch_long<2>(a, s);
  if (rb <= 4) return launch_long<4>(a, s);
  return launch_long<8>(a, s);
}

}  // namespace adapter
}  // namespace moe
