// Low-rank adapters of many requests beside a shared projection, forward and backward.
//
//   u = s (x A^T)              y = round(x W + u B)
//   v = s (dy B^T)             dx = round(dy W^T + v A)
//   dA = sum_t v_t^T x_t       dB = sum_t u_t^T dy_t
// with an adapter (A [r, d], B [r, n], s) or none for every segment of token rows.  u and v
// are fp32; they enter the products of fp32 results with all their bits, those of bf16 results with 16.
//
// Four kernels serve both directions (A and B, d and n, x and dy change places):
//   shrink       u of segments of few rows against the r rows of one table, reduction over the
//                long side;
//   shrink_long  u of segments of many rows (adapter_shrink.cu);
//   project      y: the projection on the tensor cores, the adapter's part added before the one
//                rounding (adapter_project.cuh);
//   grads        dA, dB: the sums over an adapter's tokens (adapter_grads.cu).
#include "adapter.cuh"

namespace moe {
namespace adapter {
namespace {

// --------------------------------- shrink ------------------------------------
//
// Segments of few rows (longer ones: adapter_shrink.cu).  A CTA takes a piece of 8 NB rows of
// one segment; where there are more than kPieceSegs segments, a tile of 8 NB rows holds runs of
// rows with one adapter, and CTA j of a tile (blockIdx.y) takes its runs j, j + J, ... (finding a
// piece takes a look at the segments in front of it).  The table's rows are the M operand, the tokens N = 8 at a time, so a run
// of one token costs one column block and nothing is shared between runs.  Both operands come
// from global memory as 16 bytes a lane: lane t of a row takes values 8t .. 8t+7 of 32, and the
// MMA's slots are dealt from those in the same order on both sides (a sum does not mind the order
// of its terms).  The warps split the reduction (a cluster too, where there are few CTAs).

constexpr int kShrinkWarps = 8;

template <int MB, int NB>
struct Shrink {
  static constexpr int kRankGroups = MB > 4 ? 2 : 1;  // warps that share the rows of the table
  static constexpr int kMB = MB / kRankGroups;
  static constexpr int kSlices = kShrinkWarps / kRankGroups;  // of the reduction
  static constexpr int kRows = 8 * NB;
  static constexpr int kPitch = kRows + 2;  // of a row of sums: consecutive ones in other banks
  static constexpr int kElems = 16 * MB * kPitch;
  static constexpr int kSmem = kSlices * kElems * 4 + kElems * 4;
  // 32-value pieces a warp loads at once: about a dozen 16-byte loads a lane
  static constexpr int kAhead = kMB == 1 ? (NB == 1 ? 4 : 2) : kMB == 2 ? (NB == 1 ? 3 : 2) : NB == 1 ? 2 : 1;
};

constexpr int kPieceSegs = 2048;

template <int MB, int NB>
__global__ void __launch_bounds__(32 * kShrinkWarps, 2)
shrink_kernel(const ShrinkArgs a, int split, int pieces_mode) {
  using P = Shrink<MB, NB>;
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  extern __shared__ float s_part[];            // [kSlices][16 MB][kPitch]
  float* s_sum = s_part + P::kSlices * P::kElems;  // [16 MB][kPitch]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int group = warp % P::kRankGroups, slice = warp / P::kRankGroups;
  const int m0 = group * P::kMB * 16;
  const int pieces = (a.K + 31) / 32;
  const int c0 = rank * pieces / split, c1 = (rank + 1) * pieces / split;

  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0) check_segments(a.seg, a.dev_status);

  // runs of the tile: every warp finds them for itself
  int row0 = static_cast<int>(blockIdx.x) / split * P::kRows, id;
  const uint32_t in_tile = P::kRows == 32 ? kAll : (1u << P::kRows) - 1;
  if (pieces_mode) {
    const Piece p = piece_of<32 * kShrinkWarps>(a.seg, static_cast<int>(blockIdx.x) / split, P::kRows);
    row0 = p.row;
    id = lane < p.rows ? p.adapter : kOutside;
  } else {
    id = row_adapters(a.seg, row0, lane);
  }
  if (blockIdx.y == 0 && rank == 0) {
    uint32_t none = __ballot_sync(kAll, id == kNone) & in_tile;
    for (; none != 0; none &= none - 1)
      if (static_cast<int>(threadIdx.x) < a.r)
        a.u[static_cast<int64_t>(row0 + __ffs(none) - 1) * a.r + threadIdx.x] = 0.0f;
  }
  const int before = __shfl_up_sync(kAll, id, 1);
  uint32_t starts = __ballot_sync(kAll, id >= 0 && (lane == 0 || id != before)) & in_tile;
  const uint32_t held = __ballot_sync(kAll, id >= 0) & in_tile;
  for (int nth = 0; starts != 0; ++nth) {
    const int b = __ffs(starts) - 1;  // rows b .. e - 1 of the tile
    starts &= starts - 1;
    const uint32_t stops = (starts | ~held) & ~((2u << b) - 1);  // later starts, rows without one
    const int e = min(stops != 0 ? __ffs(stops) - 1 : 32, P::kRows);
    if (nth % static_cast<int>(gridDim.y) != static_cast<int>(blockIdx.y)) continue;
    const int adapter = __shfl_sync(kAll, id, b);
    float acc[P::kMB][NB][4];
#pragma unroll
    for (int i = 0; i < P::kMB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;
    const uint16_t* tab = a.table + (static_cast<int64_t>(adapter) * a.r + m0 + g) * a.K;
    const uint16_t* xr = a.x + (row0 + g) * a.x_stride;
    for (int c = c0 + slice; c < c1; c += P::kSlices * P::kAhead) {
      uint4 xv[P::kAhead][NB], tv[P::kAhead][P::kMB][2];
#pragma unroll
      for (int h = 0; h < P::kAhead; ++h) {
        const int k = (c + h * P::kSlices) * 32 + 8 * t4;
        const bool in = c + h * P::kSlices < c1 && k < a.K;  // K is a multiple of 8
#pragma unroll
        for (int j = 0; j < NB; ++j)
          xv[h][j] = in && 8 * j + g >= b && 8 * j + g < e
                         ? __ldg(reinterpret_cast<const uint4*>(xr + 8 * j * a.x_stride + k))
                         : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < P::kMB; ++i)
#pragma unroll
          for (int o = 0; o < 2; ++o)
            tv[h][i][o] = in && m0 + 16 * i + 8 * o + g < a.r
                              ? __ldg(reinterpret_cast<const uint4*>(
                                    tab + static_cast<int64_t>(16 * i + 8 * o) * a.K + k))
                              : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int h = 0; h < P::kAhead; ++h)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          if (8 * j < e && 8 * j + 8 > b) {
#pragma unroll
            for (int i = 0; i < P::kMB; ++i) {
              const uint4 lo = tv[h][i][0], hi = tv[h][i][1];
              mma_16816(acc[i][j], lo.x, hi.x, lo.y, hi.y, xv[h][j].x, xv[h][j].y);
              mma_16816(acc[i][j], lo.z, hi.z, lo.w, hi.w, xv[h][j].z, xv[h][j].w);
            }
          }
    }
    // the slices of this CTA, then those of the cluster, in order
    float* mine = s_part + slice * P::kElems;
#pragma unroll
    for (int i = 0; i < P::kMB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (8 * j < e && 8 * j + 8 > b) {
          const int m = m0 + 16 * i + g, n = 8 * j + 2 * t4;
          *reinterpret_cast<float2*>(mine + m * P::kPitch + n) = make_float2(acc[i][j][0], acc[i][j][1]);
          *reinterpret_cast<float2*>(mine + (m + 8) * P::kPitch + n) =
              make_float2(acc[i][j][2], acc[i][j][3]);
        }
    __syncthreads();
    const float scale = __ldg(a.scale + adapter);
    const int n = (e - b) * a.r;
    if (split > 1) {
      for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int at = i % a.r * P::kPitch + b + i / a.r;
        float v = s_part[at];
#pragma unroll
        for (int s = 1; s < P::kSlices; ++s) v += s_part[s * P::kElems + at];
        s_sum[at] = v;
      }
      cluster_sync();
    }
    for (int i = rank * blockDim.x + threadIdx.x; i < n; i += split * blockDim.x) {
      const int row = b + i / a.r, m = i % a.r;
      const int at = m * P::kPitch + row;
      float v = 0.0f;
      if (split > 1) {
        v = sum_of_ranks(smem_u32(s_sum + at), split);
      } else {
#pragma unroll
        for (int s = 0; s < P::kSlices; ++s) v += s_part[s * P::kElems + at];
      }
      a.u[static_cast<int64_t>(row0 + row) * a.r + m] = scale * v;
    }
    if (split > 1) cluster_sync();  // before the sums are written again, or given up
    else __syncthreads();
  }
}

// ------------------------------- host side -----------------------------------

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <int MB, int NB>
moe_status launch_shrink_as(const ShrinkArgs& a, cudaStream_t s) {
  using P = Shrink<MB, NB>;
  auto kern = shrink_kernel<MB, NB>;
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, P::kSmem, mu, done)) return MOE_ERR_CUDA;
  // The reduction is split over a cluster where the CTAs that have work do not fill the SMs twice.
  const int64_t tiles = ceil_div(a.seg.T, P::kRows), sms = sm_count(), n_seg = a.seg.n_seg;
  const bool pieces = n_seg <= kPieceSegs;
  const int64_t grid = pieces ? tiles + n_seg : tiles;
  const int64_t J = pieces ? 1 : std::min<int64_t>(P::kRows, ceil_div(2 * n_seg, tiles));
  const int split = pow2_at_most(std::min<int64_t>(2 * sms / (grid * J), a.K / 256), 8);
  launch_clustered(kern, dim3(static_cast<unsigned>(grid * split), static_cast<unsigned>(J)),
                   32 * kShrinkWarps, P::kSmem, split, s, a, split, static_cast<int>(pieces));
  return launch_status();
}

moe_status launch_shrink(const ShrinkArgs& a, cudaStream_t s) {
  // Rows of a segment on average: from 32 on tiles of 128 rows by the tensor memory accelerator
  if (a.seg.T >= 32 * static_cast<int64_t>(a.seg.n_seg)) return shrink_long(a, s);
  const bool narrow = a.seg.T <= 256;
  const int mb = (a.r + 15) / 16;
  if (mb == 1) return narrow ? launch_shrink_as<1, 1>(a, s) : launch_shrink_as<1, 4>(a, s);
  if (mb == 2) return narrow ? launch_shrink_as<2, 1>(a, s) : launch_shrink_as<2, 4>(a, s);
  if (mb <= 4) return narrow ? launch_shrink_as<4, 1>(a, s) : launch_shrink_as<4, 4>(a, s);
  return narrow ? launch_shrink_as<8, 1>(a, s) : launch_shrink_as<8, 4>(a, s);
}

// The shape of the projection.  Up to 64 tokens: narrow tiles, the reduction shared by up to
// four CTAs until the SMs are full (one token: 16 tiles of 7168 x 128 on one / two / four CTAs each
// 36.9 / 22.7 / 14.4 us; 64 tokens of as many adapters, 2048 x 2048: 19.3 / 15.4 / 13.6).
// Above, what takes fewer cycles: a stage of 64 takes 575 in either shape (it has 32 KB a CTA), the
// adapters' part and the stores 18,000 a tile of a pair, behind the last tile or where a tile's
// MMAs are shorter, and 8,000 of 128 x 128.  Measured, flat / pair (us): 256 tokens, 4096 x 4096: 22.4
// / 34.1; 512: 29.7 / 33.0; 1,024 (r 64): 52.0 / 48.8; 1,024, 2048 x 2048: 19.3 / 21.4; 2,048: 31.2 /
// 26.7; 4,096, 2048 x 1024: 33.0 / 28.7, 768 x 2048: 30.5 / 29.3.  Where segments have few rows flat
// tiles make the adapters' part beside the MMAs: 1,000 tokens in 70 segments, 4096 x 4096: 73 / 81.
moe_status launch_project(const ProjectArgs& a, const Operands& o, bool kmaj, cudaStream_t s) {
  const int64_t sms = sm_count(), cols = ceil_div(a.N, 128);
  const int T = a.seg.T;
  if (T <= 64) {
    const int split = pow2_at_most(std::min(sms / cols, ceil_div(a.K, 128)), 4);
    return kmaj ? project_flat64_kmaj(a, o, split, s) : project_flat64(a, o, split, s);
  }
  const int64_t steps = ceil_div(a.K, 64), tiles = cols * ceil_div(T, 128);
  const int split = pow2_at_most(std::min(sms / tiles, steps), 4);
  const int64_t flat = ceil_div(tiles * split, sms) * std::max<int64_t>(575 * ceil_div(steps, split), 8000) + 6000;
  const int64_t pair_tiles = ceil_div(a.N, 256) * ceil_div(T, 256);
  const int64_t pair = ceil_div(pair_tiles, sms / 2) * std::max<int64_t>(575 * steps, 18000) + 18000;
  if (!a.y_fp32 && T >= 32 * static_cast<int64_t>(a.seg.n_seg) && pair < flat)
    return project_pair(a, o, kmaj, s);
  return kmaj ? project_flat128_kmaj(a, o, split, s) : project_flat128(a, o, split, s);
}

constexpr int64_t kMaxStride = int64_t(1) << 31;

// Sizes, strides and types of one call.
moe_status check_params(const moe_adapter_params* p) {
  if (p == nullptr || p->T < 0 || p->d <= 0 || p->n <= 0 || p->r <= 0 || p->n_adapters <= 0 ||
      p->n_seg <= 0 || p->x_stride < p->d || p->y_stride < p->n ||
      (p->y_type != MOE_DTYPE_BF16 && p->y_type != MOE_DTYPE_FP32))
    return MOE_ERR_INVALID_ARG;
  if (p->d % 8 != 0 || p->n % 8 != 0 || p->r % 8 != 0 || p->d > 65536 || p->n > 65536 ||
      p->r > 128 || p->n_adapters > 65535 || p->n_seg > 65535 || p->T > INT32_MAX - 1024 ||
      p->x_stride % 8 != 0 || p->y_stride % 8 != 0 || p->x_stride > kMaxStride ||
      p->y_stride > kMaxStride)
    return MOE_ERR_UNSUPPORTED;
  // tile numbers are 32-bit
  if (ceil_div(p->T, 8) * ceil_div(std::max(p->d, p->n), 128) >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_tables(const moe_adapter_params* p, const int32_t* seg_offsets,
                        const int32_t* seg_adapter, const void* x, const void* w, const void* a,
                        const void* b, const float* scale, const float* u) {
  if (seg_adapter == nullptr || (seg_offsets == nullptr && p->n_seg != 1) || x == nullptr ||
      w == nullptr || a == nullptr || b == nullptr || scale == nullptr || u == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(a) || !aligned16(b) || !aligned16(u) ||
      !aligned4(scale) || !aligned4(seg_offsets) || !aligned4(seg_adapter))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

Segments segments_of(const moe_adapter_params* p, const int32_t* seg_offsets,
                     const int32_t* seg_adapter) {
  return Segments{seg_offsets, seg_adapter, p->n_seg, p->T, p->n_adapters};
}

}  // namespace
}  // namespace adapter
}  // namespace moe

using namespace moe;
using namespace moe::adapter;

MOE_API moe_status moe_adapter_project(const moe_adapter_params* p, const int32_t* seg_offsets,
                                       const int32_t* seg_adapter, const moe_bf16* x,
                                       const moe_bf16* w, const moe_bf16* a, const moe_bf16* b,
                                       const float* scale, float* u, void* y,
                                       uint32_t* dev_status, moe_stream_t stream) {
  moe_status st = check_params(p);
  if (st != MOE_OK || p->T == 0) return st;
  st = check_tables(p, seg_offsets, seg_adapter, x, w, a, b, scale, u);
  if (st != MOE_OK) return st;
  if (y == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y)) return MOE_ERR_UNSUPPORTED;
  const Segments seg = segments_of(p, seg_offsets, seg_adapter);
  const cudaStream_t s = as_cuda(stream);
  st = launch_shrink(ShrinkArgs{seg, p->d, p->r, x, p->x_stride, a, scale, u, dev_status}, s);
  if (st != MOE_OK) return st;
  return launch_project(ProjectArgs{seg, p->d, p->n, p->r, u, b, y, p->y_stride,
                                           p->y_type == MOE_DTYPE_FP32, 0, 0, 0, 0, dev_status},
                               Operands{x, p->x_stride, w}, false, s);
}

MOE_API size_t moe_adapter_project_backward_workspace_size(const moe_adapter_params* p) {
  if (check_params(p) != MOE_OK) return 0;
  return std::max<size_t>(static_cast<size_t>(p->T) * p->r * 4, 16);  // v
}

MOE_API moe_status moe_adapter_project_backward(
    const moe_adapter_params* p, const int32_t* seg_offsets, const int32_t* seg_adapter,
    const moe_bf16* x, const moe_bf16* w, const moe_bf16* a, const moe_bf16* b, const float* scale,
    const float* u, const moe_bf16* dy, moe_bf16* dx, float* da, float* db, int32_t accumulate,
    void* ws, size_t ws_bytes, uint32_t* dev_status, moe_stream_t stream) {
  moe_status st = check_params(p);
  if (st != MOE_OK) return st;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (dx == nullptr && da == nullptr && db == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dx) || !aligned16(da) || !aligned16(db)) return MOE_ERR_UNSUPPORTED;
  const cudaStream_t s = as_cuda(stream);
  if (p->T == 0) {  // no tokens: zero gradients
    if (accumulate) return MOE_OK;
    if (da != nullptr && cudaMemsetAsync(da, 0, size_t(4) * p->n_adapters * p->r * p->d, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (db != nullptr && cudaMemsetAsync(db, 0, size_t(4) * p->n_adapters * p->r * p->n, s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  st = check_tables(p, seg_offsets, seg_adapter, x, w, a, b, scale, u);
  if (st != MOE_OK) return st;
  if (dy == nullptr || ws == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(ws)) return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < moe_adapter_project_backward_workspace_size(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const Segments seg = segments_of(p, seg_offsets, seg_adapter);
  float* v = static_cast<float*>(ws);
  if (dx != nullptr || da != nullptr) {
    st = launch_shrink(ShrinkArgs{seg, p->n, p->r, dy, p->y_stride, b, scale, v, dev_status}, s);
    if (st != MOE_OK) return st;
  }
  if (dx != nullptr) {
    st = launch_project(ProjectArgs{seg, p->n, p->d, p->r, v, a, dx, p->d, 0, 0, 0, 0, 0, dev_status},
                              Operands{dy, p->y_stride, w}, true, s);
    if (st != MOE_OK) return st;
  }
  if (da != nullptr || db != nullptr)
    return table_grads(GradArgs{seg,
                                p->r,
                                {{da != nullptr ? p->d : 0, v, x, p->x_stride, da},
                                 {db != nullptr ? p->n : 0, u, dy, p->y_stride, db}},
                                accumulate,
                                dx == nullptr && da == nullptr,  // (no shrink)
                                dev_status},
                       s);
  return MOE_OK;
}
