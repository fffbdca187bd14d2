// Low-rank adapters of many requests beside a shared projection, forward and backward.
//
//   u = s (x A^T)              y = round(x W + u B)
//   v = s (dy B^T)             dx = round(dy W^T + v A)
//   dA = sum_t v_t^T x_t       dB = sum_t u_t^T dy_t
// with an adapter (A [r, d], B [r, n], s) or none for every segment of token rows.  u and v
// are fp32, so an adapter's part of y is as exact as the projection itself.
//
// Three kernels serve both directions (A and B, d and n, x and dy change places):
//   shrink   u: rows against the r rows of one table, reduction over the long side.
//   project  y: the projection on the tensor cores, the adapter's part added before the one
//            rounding.
//   grads    dA, dB: the sums over an adapter's tokens.
#include <algorithm>

#include "smem.cuh"
#include "umma.cuh"

namespace moe {
namespace {

struct Segments {
  const int32_t* offsets;  // [n_seg + 1], or nullptr: one segment of all rows
  const int32_t* adapter;  // [n_seg]
  int n_seg, T, n_adapters;
};

constexpr int kOutside = -2;  // a row of no segment
constexpr int kNone = -1;     // a segment without an adapter

__device__ __forceinline__ int seg_begin(const Segments& s, int q) {
  return s.offsets == nullptr ? (q == 0 ? 0 : s.T) : __ldg(s.offsets + q);
}

// Rows [b, e) of segment q inside [0, T); empty where the offsets are out of order.
__device__ __forceinline__ void seg_rows(const Segments& s, int q, int& b, int& e) {
  b = max(seg_begin(s, q), 0);
  e = min(seg_begin(s, q + 1), s.T);
}

// Adapter of segment q; an id outside the tables counts as none.
__device__ __forceinline__ int seg_adapter(const Segments& s, int q) {
  const int a = __ldg(s.adapter + q);
  return a >= 0 && a < s.n_adapters ? a : kNone;
}

// Adapter of row row0 + lane (kNone, or kOutside), by a whole warp: a search that asks 32
// segments at a time for the one that holds row0 (a binary one would be as many loads one after
// the other as it has steps), then the ends of the segments behind it, 32 at a time.
__device__ __forceinline__ int row_adapters(const Segments& s, int row0, int lane) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  int lo = 0, n = s.n_seg;  // the last segment that starts at or before row0 is in [lo, lo + n)
  while (n > 1) {
    const int stride = (n + 31) / 32;
    const int q = lo + lane * stride;
    const bool at = lane * stride < n && seg_begin(s, q) <= row0;
    const int c = __popc(__ballot_sync(kAll, at));  // ordered offsets: the first c of them
    const int skip = c > 0 ? (c - 1) * stride : 0;
    lo += skip;
    n = min(stride, n - skip);
  }
  const int row = row0 + lane;
  const bool before = row < seg_begin(s, lo);  // (in front of the first segment)
  int seg = -1;
  for (int q0 = lo; q0 < s.n_seg; q0 += 32) {
    const int end = q0 + lane < s.n_seg ? seg_begin(s, q0 + lane + 1) : 0x7FFFFFFF;
    int c = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) c += __shfl_sync(kAll, end, i) <= row;
    if (seg < 0 && c < 32) seg = q0 + c;
    if (__all_sync(kAll, seg >= 0)) break;
  }
  if (row >= s.T || before || seg < 0 || seg >= s.n_seg) return kOutside;
  // (offsets out of order may name a segment that does not hold the row: still inside the table)
  return seg_adapter(s, seg);
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 blocks of 16-bit values, transposed; lane l gives the address of row l % 8 of block
// l / 8.
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// --------------------------------- shrink ------------------------------------
//
// A tile of 8 NB rows holds runs of rows with one adapter; CTA j of a tile (blockIdx.y) takes its
// runs j, j + J, ...  The table's rows are the M operand, the tokens N = 8 at a time, so a run
// of one token costs one column block and nothing is shared between runs.  Both operands come
// from global memory as 16 bytes a lane: lane t of a row takes values 8t .. 8t+7 of 32, and the
// MMA's slots are dealt from those in the same order on both sides (a sum does not mind the order
// of its terms).  The warps split the reduction (a cluster too, where there are few CTAs).

constexpr int kShrinkWarps = 8;

struct ShrinkArgs {
  Segments seg;
  int K, r;
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* table;  // [n_adapters, r, K]
  const float* scale;     // [n_adapters]
  float* u;               // [T, r]
  uint32_t* dev_status;
};

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

template <int MB, int NB>
__global__ void __launch_bounds__(32 * kShrinkWarps, 2)
shrink_kernel(const ShrinkArgs a, int split) {
  using P = Shrink<MB, NB>;
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  extern __shared__ float s_part[];            // [kSlices][16 MB][kPitch]
  float* s_sum = s_part + P::kSlices * P::kElems;  // [16 MB][kPitch]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int row0 = static_cast<int>(blockIdx.x) / split * P::kRows;
  const int group = warp % P::kRankGroups, slice = warp / P::kRankGroups;
  const int m0 = group * P::kMB * 16;
  const int pieces = (a.K + 31) / 32;
  const int c0 = rank * pieces / split, c1 = (rank + 1) * pieces / split;

  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // the segment table, looked over once
    for (int q = threadIdx.x; q < a.seg.n_seg; q += blockDim.x) {
      const int b = seg_begin(a.seg, q), e = seg_begin(a.seg, q + 1);
      if (b < 0 || e < b || e > a.seg.T) report(a.dev_status, MOE_DEV_BAD_MAP);
      const int id = __ldg(a.seg.adapter + q);
      if (id < kNone || id >= a.seg.n_adapters) report(a.dev_status, MOE_DEV_BAD_ADAPTER);
    }
  }

  // runs of the tile: every warp finds them for itself
  const int id = row_adapters(a.seg, row0, lane);
  const uint32_t in_tile = P::kRows == 32 ? kAll : (1u << P::kRows) - 1;
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
        const uint32_t addr = smem_u32(s_sum + at);
        for (int o = 0; o < split; ++o) v += ld_cluster(map_to_rank(addr, o));
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

// --------------------------------- project -----------------------------------
//
// D^T = W^T X^T: the weight's columns are the M operand, the tokens N, so a decode batch is a
// narrow tile and the weight streams once.  Roles of the 352 threads:
//   warp 0       TMA producer: [64 k x 128] of the weight (16 KB) and [tokens x 64 k] of x
//   warp 1       tensor memory; lane 0 issues four MMAs (K = 16) a stage
//   warps 2..9   epilogue: warp (quad, sub) has the 16 weight columns at 32 quad + 16 sub
//   warp 10      the tile's runs of rows with one adapter, and the runs' tables by TMA
//   warp 11      u, 32 tokens at a time, by TMA
// The adapters' part is a product of mma.sync in the epilogue: u B is r / d of the work and a
// run may be one token long, where tcgen05's narrowest tile is 16 columns by 128 rows of the
// table.  tcgen05's 16x256b loads give the accumulators in mma.sync's own layout, 16 weight
// columns by 8 tokens at a time, so a run's table (transposed by ldmatrix into registers, once a
// run) is multiplied with the u of the 8 tokens onto the sums themselves.  Where several runs
// meet in 8 tokens every column takes the result of its own run: nothing of one request, not
// even 0 times an infinity, reaches another's rows.  u enters as two bf16 numbers.
//
// Shapes (choose_shape has the rule):
//   pair   a cluster of two CTAs, 256 weight columns by 256 tokens (cta_group::2), two
//          accumulator buffers that fill the tensor memory
//   flat   one CTA, 128 weight columns by TN = 64 or 128 tokens; the adapters' part is made
//          while the MMAs run and waits in tensor memory.  S > 1: a cluster shares a tile, each
//          CTA a part of the reduction; the CTA of rank c finishes its S-th of the tokens and
//          gets the others' sums through distributed shared memory.
// fp32 results of long reductions are summed in pieces of kPiece: the tensor cores' own fp32
// sums lose 2^-26 a step (7168: 8e-6 of the result, in pieces of 1024 1e-6).
// The weight, x and the tables are staged before shrink has ended; u is waited for.

struct ProjectArgs {
  Segments seg;
  int K, N, r;
  const float* u;  // [T, r]
  void* y;
  int64_t y_stride;
  int y_fp32;
  int n_blocks, t_blocks, n_inner;
  int x_rows;   // rows of a box of x: those behind the batch's last are never staged
  int slots;    // of the tables
  int u_slots;
  uint32_t* dev_status;
};

constexpr int kThreads = 384;
constexpr int kWBytes = 128 * 64 * 2;
constexpr int kWBox = 64 * 64 * 2;
constexpr int kPiece = 16;      // steps of 64 to a piece of an fp32 result's reduction
constexpr int kMaxSlots = 16;
constexpr int kUBox = 32 * 32 * 4;  // [32 tokens][32 of r] fp32
constexpr int kMaxRank = 128;

template <int TN, int S, int CG>
struct Shape {
  static constexpr int kStageBytes = kWBytes + TN / CG * 128;
  static constexpr int kStages = CG == 2 ? 5 : TN == 128 ? (S == 2 ? 4 : 3) : S == 1 ? 5 : 4;
  static constexpr int kOwn = TN / S;
  // 64 KB of tables on their way where runs may be single tokens (32 KB: 128 tokens of as many
  // adapters took a third longer)
  static constexpr int kTableBytes = (CG == 2 || (TN == 128 && (S == 2 || S == 8)) ? 32 : 64) * 1024;
  static constexpr int kUBytes = (S >= 4 ? 16 : 32) * 1024;
  static constexpr int kRedBytes = (S - 1) * kOwn * 512;  // [S - 1][kOwn / 8][8][32] float4
  // full[st], empty[st], tfull[2], tempty[2], jfull[2], jempty[2], tbfull[], tbempty[], ufull[],
  // uempty[], red, drain
  static constexpr int kBars = 2 * kStages + 8 + 4 * kMaxSlots + 2;
  static constexpr int kTmem = CG == 2 ? 2 * TN : 4 * TN;  // two buffers, (flat) the sums
  static constexpr int kSmem =
      1024 + kStages * kStageBytes + kTableBytes + kUBytes + kRedBytes + kBars * 8 + 2 * kOwn * 2 + 2 * (kOwn / 8) * 4 + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kOwn % 8 == 0 && kTmem <= 512, "shape");
  static_assert(kTableBytes >= 256 * kMaxRank, "one table at least");
  static_assert(kUBytes >= (kOwn > 32 ? 2 : 1) * kUBox * kMaxRank / 32, "two pieces of u where there are");
};

// The table of one run in registers, and its place in the ring.
struct Table {
  uint32_t f[kMaxRank / 16][4];
  int run;        // whose table f holds
  int slot;
  uint32_t ph;
};

// Stores 16 weight columns from n by 8 tokens from row (the layout of umma_ld_frag).
__device__ __forceinline__ void put_frag(const ProjectArgs& a, const float (&c)[4], int row, int n,
                                         const int16_t* run, int lane) {
  const int g = lane >> 2, t4 = lane & 3;
  if (a.y_fp32) {
    float* y = static_cast<float*>(a.y) + static_cast<int64_t>(row) * a.y_stride + n + g;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (run[2 * t4 + e] != kOutside) {
        if (n < a.N) y[(2 * t4 + e) * a.y_stride] = c[e];
        if (n + 8 < a.N) y[(2 * t4 + e) * a.y_stride + 8] = c[2 + e];
      }
    return;
  }
  // rows become tokens: two 8 x 8 blocks transposed, then 4 columns to a lane
  uint32_t d0 = pack_bf16x2(c[0], c[1]), d1 = pack_bf16x2(c[2], c[3]);
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(d0));
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(d1));
  const bool odd = t4 & 1;
  const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? d0 : d1, 1);
  const int col = n + (odd ? 8 + 2 * (t4 - 1) : 2 * t4);
  if (col < a.N && run[g] != kOutside)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + static_cast<int64_t>(row + g) * a.y_stride +
                              col) = odd ? make_uint2(other, d1) : make_uint2(d0, other);
}

template <int TN, int S, int CG, bool KMAJ>
__global__ void __launch_bounds__(kThreads, 1)
project_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
               const __grid_constant__ CUtensorMap map_t, const __grid_constant__ CUtensorMap map_u,
               const ProjectArgs a) {
  using F = Shape<TN, S, CG>;
  static_assert(CG == 1 || S == 1, "one kind of cluster");
  constexpr int kStages = F::kStages, kOwn = F::kOwn;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stage_base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_table = stage_base + kStages * F::kStageBytes;
  uint8_t* s_u = s_table + F::kTableBytes;
  uint8_t* s_red = s_u + F::kUBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_red + F::kRedBytes);
  int16_t* s_run = reinterpret_cast<int16_t*>(bars + F::kBars);  // [2][kOwn]: run of a token
  // [2][kOwn / 8]: first run of 8 tokens, and in the high half the last one (-1: none)
  int* s_span = reinterpret_cast<int*>(s_run + 2 * kOwn);
  volatile int* abort_flag = s_span + 2 * (kOwn / 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_span + 2 * (kOwn / 8)) + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kCluster = S * CG;
  const int rank = kCluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const bool leader = CG == 1 || rank == 0;
  const int first = static_cast<int>(blockIdx.x) / kCluster;
  const int step = static_cast<int>(gridDim.x) / kCluster;
  const int total = a.n_blocks * a.t_blocks;
  const int steps = (a.K + 63) / 64;
  const int k0 = S > 1 ? rank * steps / S : 0, k1 = S > 1 ? (rank + 1) * steps / S : steps;
  const int piece = CG == 1 && a.y_fp32 ? kPiece : steps;
  const int rp = (a.r + 15) & ~15;
  const int own0 = S > 1 ? rank * kOwn : 0;  // this CTA's tokens of the tile
  const int u_bytes = (a.r + 31) / 32 * kUBox;  // a piece of u
  const uint32_t stage_tx = kWBytes + a.x_rows * 128;

  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + kStages + s); };
  auto tfull_bar = [&](int b) { return smem_u32(bars + 2 * kStages + b); };
  auto tempty_bar = [&](int b) { return smem_u32(bars + 2 * kStages + 2 + b); };
  auto jfull_bar = [&](int b) { return smem_u32(bars + 2 * kStages + 4 + b); };
  auto jempty_bar = [&](int b) { return smem_u32(bars + 2 * kStages + 6 + b); };
  auto tbfull_bar = [&](int s) { return smem_u32(bars + 2 * kStages + 8 + s); };
  auto tbempty_bar = [&](int s) { return smem_u32(bars + 2 * kStages + 8 + kMaxSlots + s); };
  auto ufull_bar = [&](int s) { return smem_u32(bars + 2 * kStages + 8 + 2 * kMaxSlots + s); };
  auto uempty_bar = [&](int s) { return smem_u32(bars + 2 * kStages + 8 + 3 * kMaxSlots + s); };
  const uint32_t red_bar = smem_u32(bars + 2 * kStages + 8 + 4 * kMaxSlots);
  const uint32_t drain_bar = red_bar + 8;
  // first token and first weight column of this CTA's part of tile t
  auto tile = [&](int t, int& row0, int& n0) {
    const int nb = a.n_inner ? t % a.n_blocks : t / a.t_blocks;
    const int tb = a.n_inner ? t / a.n_blocks : t % a.t_blocks;
    row0 = tb * TN;
    n0 = nb * 128 * CG + (CG == 2 ? rank * 128 : 0);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 8 * CG);  // one arrival per epilogue warp
      mbar_init(jfull_bar(b), 1);
      mbar_init(jempty_bar(b), 8);
    }
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(tbfull_bar(s), 1);
      mbar_init(tbempty_bar(s), 8);
      mbar_init(ufull_bar(s), 1);
      mbar_init(uempty_bar(s), 8);
    }
    mbar_init(red_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (S > 1) mbar_arrive_expect_tx(red_bar, F::kRedBytes);
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_t)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_u)) : "memory");
  }
  if (warp == 1) {
    if constexpr (CG == 2) umma_alloc_pair(smem_u32(tmem_slot), F::kTmem);
    else umma_alloc(smem_u32(tmem_slot), F::kTmem);
  }
  umma_fence_before();
  __syncthreads();
  if constexpr (kCluster > 1) cluster_sync();  // the partners' barriers are initialised
  umma_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool awaited = false;

  if (warp == 0) {
    if (lane == 0) {
      // ---- TMA producer ----
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        int row0, n0;
        tile(t, row0, n0);
        if (CG == 2) row0 += rank * (TN / 2);
        for (int k = k0; k < k1; ++k) {
          if (!wait_bounded(empty_bar(s), ph ^ 1u, abort_flag, a.dev_status)) { ok = false; break; }
          const uint32_t st = smem_u32(stage_base + s * F::kStageBytes);
          if constexpr (CG == 2) {
            const uint32_t bar = map_to_rank(full_bar(s), 0);
            if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * stage_tx);
            if (KMAJ) {
              tma_load_2d_pair(st, &map_w, bar, k * 64, n0);
            } else {
              tma_load_2d_pair(st, &map_w, bar, n0, k * 64);
              tma_load_2d_pair(st + kWBox, &map_w, bar, n0 + 64, k * 64);
            }
            tma_load_2d_pair(st + kWBytes, &map_x, bar, k * 64, row0);
          } else {
            mbar_arrive_expect_tx(full_bar(s), stage_tx);
            if (KMAJ) {
              tma_load_2d(st, &map_w, full_bar(s), k * 64, n0);
            } else {
              tma_load_2d(st, &map_w, full_bar(s), n0, k * 64);
              tma_load_2d(st + kWBox, &map_w, full_bar(s), n0 + 64, k * 64);
            }
            tma_load_2d(st + kWBytes, &map_x, full_bar(s), k * 64, row0);
          }
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
      if (!ok) {  // copies in flight land before the shared memory is given up
        if (leader) {
          for (int i = 0; i < kStages; ++i) {
            if (--s < 0) { s = kStages - 1; ph ^= 1u; }
            wait_drain(full_bar(s), ph);
          }
        } else {  // they are counted on the leader's barriers: a fixed window
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < 2000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---- MMA issuer ----
      constexpr uint32_t idesc = umma_idesc_bf16(128 * CG, TN, !KMAJ);
      int s = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true, issued = false;
      for (int t = first; t < total && ok; t += step) {
        for (int kp = k0; kp < k1 && ok; kp += piece) {
          if (!wait_bounded(tempty_bar(buf), acc_ph ^ 1u, abort_flag, a.dev_status)) { ok = false; break; }
          umma_fence_after();
          const int ke = min(kp + piece, k1);
          for (int k = kp; k < ke; ++k) {
            if (!wait_bounded(full_bar(s), ph, abort_flag, a.dev_status)) { ok = false; break; }
            umma_fence_after();
            const uint32_t st = smem_u32(stage_base + s * F::kStageBytes);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t ad = KMAJ ? umma_desc(st + kk * 32) : umma_desc_mn(st + kk * 16 * 128, kWBox);
              const uint64_t bd = umma_desc(st + kWBytes + kk * 32);
              if constexpr (CG == 2) umma_bf16_pair(tmem + buf * TN, ad, bd, idesc, k > kp || kk > 0);
              else umma_bf16(tmem + buf * TN, ad, bd, idesc, k > kp || kk > 0);
            }
            issued = true;
            if constexpr (CG == 2) umma_commit_pair(empty_bar(s), 0x3);
            else umma_commit(empty_bar(s));
            if (++s == kStages) { s = 0; ph ^= 1u; }
          }
          if (!ok) break;
          if constexpr (CG == 2) umma_commit_pair(tfull_bar(buf), 0x3);
          else umma_commit(tfull_bar(buf));
          if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
        }
      }
      if (!ok && issued) {
        if constexpr (CG == 2) umma_commit_pair(drain_bar, 0x1);
        else umma_commit(drain_bar);
        wait_drain(drain_bar, 0);
      }
    }
  } else if (warp == 10) {
    // ---- runs and their tables ----
    int jb = 0, slot = 0, used = 0;
    uint32_t jph = 0, sph = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      int row0, n0;
      tile(t, row0, n0);
      constexpr int kChunks = (kOwn + 31) / 32;
      int id[kChunks];
      uint32_t starts[kChunks];
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        id[c] = row_adapters(a.seg, row0 + own0 + 32 * c, lane);
        if (32 * c + lane >= kOwn) id[c] = kOutside;
      }
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(jempty_bar(jb), jph ^ 1u, abort_flag, a.dev_status))) {
        ok = false;
        break;
      }
      int runs = 0, last = kOutside;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        int before = __shfl_up_sync(0xFFFFFFFFu, id[c], 1);
        if (lane == 0) before = last;
        last = __shfl_sync(0xFFFFFFFFu, id[c], 31);
        starts[c] = __ballot_sync(0xFFFFFFFFu, id[c] >= 0 && id[c] != before);
        const int run = runs + __popc(starts[c] & (0xFFFFFFFFu >> (31 - lane))) - 1;
        const int mine = id[c] >= 0 ? run : id[c];
        int hi = mine, lo = mine >= 0 ? mine : 0x7FFF;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
          hi = max(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
          lo = min(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        }
        if (32 * c + lane < kOwn) {
          s_run[jb * kOwn + 32 * c + lane] = static_cast<int16_t>(mine);
          if ((lane & 7) == 0) s_span[jb * (kOwn / 8) + 4 * c + lane / 8] = hi < 0 ? -1 : lo | hi << 16;
        }
        runs += __popc(starts[c]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(jfull_bar(jb));
      if (++jb == 2) { jb = 0; jph ^= 1u; }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t m = starts[c];
        while (m != 0 && ok) {
          const int e = __shfl_sync(0xFFFFFFFFu, id[c], __ffs(m) - 1);
          m &= m - 1;
          if (!__all_sync(0xFFFFFFFFu, wait_bounded(tbempty_bar(slot), sph ^ 1u, abort_flag, a.dev_status))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const uint32_t dst = smem_u32(s_table + slot * 256 * rp);
            mbar_arrive_expect_tx(tbfull_bar(slot), 256 * rp);
            tma_load_3d(dst, &map_t, tbfull_bar(slot), n0, 0, e);
            tma_load_3d(dst + 128 * rp, &map_t, tbfull_bar(slot), n0 + 64, 0, e);
          }
          ++used;
          if (++slot == a.slots) { slot = 0; sph ^= 1u; }
        }
      }
    }
    if (!ok && lane == 0)
      for (int i = 0; i < min(used, a.slots); ++i) {
        if (--slot < 0) { slot = a.slots - 1; sph ^= 1u; }
        wait_drain(tbfull_bar(slot), sph);
      }
  } else if (warp == 11) {
    if (lane == 0) {
      // ---- u ----
      pdl_wait();
      int s = 0, used = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        int row0, n0;
        tile(t, row0, n0);
        for (int j = 0; j < kOwn; j += 32) {
          if (!wait_bounded(uempty_bar(s), ph ^ 1u, abort_flag, a.dev_status)) { ok = false; break; }
          mbar_arrive_expect_tx(ufull_bar(s), u_bytes);
          for (int c = 0; c < a.r; c += 32)
            tma_load_2d(smem_u32(s_u + s * u_bytes + c / 32 * kUBox), &map_u, ufull_bar(s), c,
                        row0 + own0 + j);
          ++used;
          if (++s == a.u_slots) { s = 0; ph ^= 1u; }
        }
      }
      if (!ok)
        for (int i = 0; i < min(used, a.u_slots); ++i) {
          if (--s < 0) { s = a.u_slots - 1; ph ^= 1u; }
          wait_drain(ufull_bar(s), ph);
        }
    }
  } else {
    // ---- epilogue ----
    pdl_wait();  // (what is written here may still be read by the kernels before)
    const int quad = warp & 3, sub = (warp - 2) >> 2;
    const int g = lane >> 2, t4 = lane & 3;
    const int m0 = 32 * quad + 16 * sub;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(m0) << 16);
    const uint32_t sums = taddr + 2 * TN;  // (flat) [kOwn], or in pieces [TN]
    Table tb;
    tb.slot = 0;
    tb.ph = 0;
    int buf = 0, jb = 0, us = 0;
    uint32_t acc_ph = 0, jph = 0, uph = 0;
    // ldmatrix: this lane's row of the four 8 x 8 blocks of (16 k, 16 columns)
    const int lk = (lane & 7) + (lane & 16 ? 8 : 0), ln = m0 + (lane & 8);
    const uint32_t lm = smem_u32(s_table) + (ln >> 6) * 128 * rp + lk * 128 + ((((ln & 63) >> 3) ^ (lk & 7)) << 4);

    // The table of run j into registers, its slot given back: false if the wait gave up.
    auto take = [&](int j) {
      if (j == tb.run) return true;
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(tbfull_bar(tb.slot), tb.ph, abort_flag, a.dev_status)))
        return false;
      const uint32_t at = lm + tb.slot * 256 * rp;
#pragma unroll
      for (int k = 0; k < kMaxRank / 16; ++k)
        if (16 * k < a.r) ldmatrix_trans(tb.f[k], at + k * 2048);
      __syncwarp();
      if (lane == 0) mbar_arrive(tbempty_bar(tb.slot));
      if (++tb.slot == a.slots) { tb.slot = 0; tb.ph ^= 1u; }
      tb.run = j;
      return true;
    };
    // u of 16 ranks of a token as two bf16 numbers a value, in the layout of mma.sync's second
    // operand: w[0..1] the values, w[2..3] what their rounding left.
    auto split_u = [&](const uint8_t* row_u, int swz, int k, uint32_t (&w)[4]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int word = (16 * k) % 32 + 8 * h + 2 * t4;  // of the 32 of a row
        const float2 f = *reinterpret_cast<const float2*>(
            row_u + k / 2 * kUBox + (((word >> 2) ^ swz) << 4) + (word & 3) * 4);
        w[h] = pack_bf16x2(f.x, f.y);
        w[2 + h] = pack_bf16x2(f.x - __uint_as_float(w[h] << 16),
                               f.y - __uint_as_float(w[h] & 0xFFFF0000u));
      }
    };
    // c += u B on 8 tokens of several runs.
    auto add_runs = [&](float (&c)[4], const uint8_t* row_u, const int16_t* run, int span) {
      if (span < 0) return true;
      const int r0 = run[2 * t4], r1 = run[2 * t4 + 1];
      for (int j = span & 0xFFFF; j <= span >> 16; ++j) {
        if (!take(j)) return false;
        float d[4] = {c[0], c[1], c[2], c[3]}, e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kMaxRank / 16; ++k)
          if (16 * k < a.r) {
            uint32_t w[4];
            split_u(row_u, g, k, w);
            mma_16816(d, tb.f[k][0], tb.f[k][1], tb.f[k][2], tb.f[k][3], w[0], w[1]);
            mma_16816(e, tb.f[k][0], tb.f[k][1], tb.f[k][2], tb.f[k][3], w[2], w[3]);
          }
        if (r0 == j) { c[0] = d[0] + e[0]; c[2] = d[2] + e[2]; }
        if (r1 == j) { c[1] = d[1] + e[1]; c[3] = d[3] + e[3]; }
      }
      return true;
    };

    bool ok = true;
    for (int t = first; t < total; t += step) {
      int row0, n0;
      tile(t, row0, n0);
      const int n = n0 + m0;
      tb.run = -1;
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(jfull_bar(jb), jph, abort_flag, a.dev_status))) break;
      const int16_t* run = s_run + jb * kOwn;
      const int row_own = row0 + own0;
      if constexpr (CG == 2) {
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(tfull_bar(buf), acc_ph, abort_flag, a.dev_status))) break;
        umma_fence_after();
      }
      const int* span = s_span + jb * (kOwn / 8);
      constexpr int kGroups = kOwn < 32 ? kOwn / 8 : 4;
      for (int j = 0; j < kOwn && ok; j += 32) {
        ok = __all_sync(0xFFFFFFFFu, wait_bounded(ufull_bar(us), uph, abort_flag, a.dev_status));
        if (!ok) break;
        const uint8_t* row_u = s_u + us * u_bytes + g * 128;  // (rows of 8 i + g share g's swizzle)
        const int r0 = run[j], r1 = run[j + 8 * kGroups - 1];
        if (r0 == r1) {  // one run, or no adapter (or outside: never stored)
          ok = r0 < 0 || take(r0);
          float c[kGroups][4];
#pragma unroll
          for (int i = 0; i < kGroups; ++i) {
            if constexpr (CG == 2) {
              umma_ld_frag(taddr + buf * TN + j + 8 * i, c[i]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) c[i][e] = 0.0f;
            }
          }
          if constexpr (CG == 2) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) umma_ld_frag_wait(c[i]);
          }
          if (r0 >= 0 && ok) {
#pragma unroll
            for (int k = 0; k < kMaxRank / 16; ++k)
              if (16 * k < a.r) {
                uint32_t w[kGroups][4];
#pragma unroll
                for (int i = 0; i < kGroups; ++i) split_u(row_u + i * 1024, g, k, w[i]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int i = 0; i < kGroups; ++i)
                    mma_16816(c[i], tb.f[k][0], tb.f[k][1], tb.f[k][2], tb.f[k][3], w[i][2 * h],
                              w[i][2 * h + 1]);
              }
          }
#pragma unroll
          for (int i = 0; i < kGroups; ++i) {
            if constexpr (CG == 2) put_frag(a, c[i], row_own + j + 8 * i, n, run + j + 8 * i, lane);
            else umma_st_frag(sums + own0 + j + 8 * i, c[i]);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < kGroups && ok; ++i) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (CG == 2) {
              umma_ld_frag(taddr + buf * TN + j + 8 * i, c);
              umma_ld_frag_wait(c);
            }
            ok = add_runs(c, row_u + i * 1024, run + j + 8 * i, span[j / 8 + i]);
            if constexpr (CG == 2) put_frag(a, c, row_own + j + 8 * i, n, run + j + 8 * i, lane);
            else umma_st_frag(sums + own0 + j + 8 * i, c);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(uempty_bar(us));
        if (++us == a.u_slots) { us = 0; uph ^= 1u; }
      }
      if (!ok) break;
      if constexpr (CG == 2) {
        umma_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(map_to_rank(tempty_bar(buf), 0));
          mbar_arrive(jempty_bar(jb));
        }
        if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
      } else {
        if (S > 1 && k0 + piece < k1) {  // the other tokens' sums start at zero
          const float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int j = 0; j < TN; j += 8)
            if (j < own0 || j >= own0 + kOwn) umma_st_frag(sums + j, z);
        }
        umma_st_wait();
        int kp = k0;
        for (; kp + piece < k1; kp += piece) {  // every piece but the last onto the sums
          if (!(ok = __all_sync(0xFFFFFFFFu, wait_bounded(tfull_bar(buf), acc_ph, abort_flag, a.dev_status))))
            break;
          umma_fence_after();
          for (int j = 0; j < TN; j += 8) {
            float c[4], q[4];
            umma_ld_frag(taddr + buf * TN + j, c);
            umma_ld_frag(sums + j, q);
            umma_ld_frag_wait(c);
            umma_ld_frag_wait(q);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] += q[e];
            umma_st_frag(sums + j, c);
          }
          umma_st_wait();
          umma_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty_bar(buf));
          if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
        }
        if (!ok) break;
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(tfull_bar(buf), acc_ph, abort_flag, a.dev_status))) break;
        umma_fence_after();
        if constexpr (S > 1) {
          awaited = true;
          for (int i = 1; i < S; ++i) {  // the partners' tokens first
            const int owner = (rank + i) % S;
            const uint32_t bar = map_to_rank(red_bar, owner);
            const uint32_t dst = map_to_rank(
                smem_u32(s_red + (S - 1 - i) * kOwn * 512 + (warp - 2) * 512 + lane * 16), owner);
            for (int j = 0; j < kOwn; j += 8) {
              float c[4];
              umma_ld_frag(taddr + buf * TN + owner * kOwn + j, c);
              umma_ld_frag_wait(c);
              if (k0 + piece < k1) {
                float q[4];
                umma_ld_frag(sums + owner * kOwn + j, q);
                umma_ld_frag_wait(q);
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] += q[e];
              }
              st_async4(dst + j * 512, bar, c[0], c[1], c[2], c[3]);
            }
          }
          if (!__all_sync(0xFFFFFFFFu, wait_bounded<true>(red_bar, 0, abort_flag, a.dev_status))) break;
        }
        for (int j = 0; j < kOwn; j += 8) {
          float c[4], q[4];
          umma_ld_frag(taddr + buf * TN + own0 + j, c);
          umma_ld_frag(sums + own0 + j, q);
          umma_ld_frag_wait(c);
          umma_ld_frag_wait(q);
#pragma unroll
          for (int e = 0; e < 4; ++e) c[e] += q[e];
          if constexpr (S > 1) {
            for (int o = 0; o < S - 1; ++o) {
              const float4 p = *reinterpret_cast<const float4*>(s_red + o * kOwn * 512 + j * 512 +
                                                                (warp - 2) * 512 + lane * 16);
              c[0] += p.x; c[1] += p.y; c[2] += p.z; c[3] += p.w;
            }
          }
          put_frag(a, c, row_own + j, n, run + j, lane);
        }
        umma_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(tempty_bar(buf));
          mbar_arrive(jempty_bar(jb));
        }
        if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
      }
      if (++jb == 2) { jb = 0; jph ^= 1u; }
    }
  }

  // ---- teardown ----
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  if constexpr (kCluster > 1) {
    cluster_sync();  // no CTA leaves while a partner may still reach it
    // (after a wait that gave up: nor before the sums that were on their way)
    if (S > 1 && threadIdx.x == 64 && awaited && *abort_flag) wait_drain(red_bar, 0);
  }
  umma_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (CG == 2) umma_dealloc_pair(tmem, F::kTmem);
    else umma_dealloc(tmem, F::kTmem);
  }
  pdl_trigger();
}

// ---------------------------------- grads ------------------------------------
//
// D_a[m, k] = sum over a's tokens of p[t, m] q[t, k], p fp32 [T, r] (u or v), q bf16 (dy or x).
// A CTA takes one adapter and 128 columns (a cluster: parts of the adapter's tokens, added in
// order).  p goes into the MMA as three bf16 numbers, the value and what each rounding left, and
// every piece of kGradTokens rows is added to the sums in fp32 registers: the gradient is as
// exact as an fp32 sum.  Rows of other segments are never loaded: zeros stand in
// their place in both operands.

struct GradArgs {
  Segments seg;
  int K, r;
  const float* p;
  const uint16_t* q;
  int64_t q_stride;
  float* out;  // [n_adapters, r, K]
  int accumulate;
};

constexpr int kGradTokens = 32;
constexpr int kGradCols = 128;
constexpr int kGradStages = 4;
constexpr int kGradRow = kGradCols * 2 + 16;  // bytes of a staged row of q

template <int MB>
struct Grad {
  static constexpr int kPRow = 16 * MB * 4;         // bytes of a staged row of p
  static constexpr int kStageBytes = kGradTokens * (kGradRow + kPRow);
  static constexpr int kSplitRow = 16 * MB * 2 + 16;  // of one of the three bf16 parts of p
  static constexpr int kSplitBytes = 3 * kGradTokens * kSplitRow;
  static constexpr int kSum = 16 * MB * kGradCols * 4;
  static constexpr int kRing = kGradStages * kStageBytes + kSplitBytes;
  static constexpr int kSmem = kRing > kSum ? kRing : kSum;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}

template <int MB>
__global__ void __launch_bounds__(256)
grads_kernel(const GradArgs a, int split) {
  using P = Grad<MB>;
  extern __shared__ __align__(16) uint8_t s_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int col0 = static_cast<int>(blockIdx.x) / split * kGradCols;
  const int id = blockIdx.y;
  pdl_wait();
  pdl_trigger();

  // the adapter's tokens, in order of its segments: this CTA's part of them
  int64_t count = 0;
  for (int q0 = 0; q0 < a.seg.n_seg; q0 += 32) {
    int n = 0;
    if (q0 + lane < a.seg.n_seg && __ldg(a.seg.adapter + q0 + lane) == id) {
      int b, e;
      seg_rows(a.seg, q0 + lane, b, e);
      n = max(e - b, 0);
    }
    count += __reduce_add_sync(0xFFFFFFFFu, n);
  }
  const int64_t part0 = count * rank / split, part1 = count * (rank + 1) / split;

  float acc[MB][2][4];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;

  // The pieces of kGradTokens rows, one after the other (every warp walks the same table):
  // `next` finds the next one.
  int q = -1, b = 0, e = 0, cand = 0;
  uint32_t mask = 0;
  int q_base = -32;
  int64_t seen = 0;  // tokens of the adapter before the current segment
  auto next = [&](int& row, int& rows) {
    while (true) {
      if (b < e) {
        row = b;
        rows = min(e - b, kGradTokens);
        b += rows;
        return true;
      }
      while (mask == 0) {
        q_base += 32;
        if (q_base >= a.seg.n_seg) return false;
        cand = q_base + lane < a.seg.n_seg ? __ldg(a.seg.adapter + q_base + lane) : -1;
        mask = __ballot_sync(0xFFFFFFFFu, cand == id);
      }
      q = q_base + __ffs(mask) - 1;
      mask &= mask - 1;
      seg_rows(a.seg, q, b, e);
      if (e <= b) { e = b; continue; }
      const int n = e - b;
      const int64_t from = part0 > seen ? part0 - seen : 0, to = part1 - seen;
      seen += n;
      e = b + static_cast<int>(to < n ? (to > 0 ? to : 0) : n);
      b += static_cast<int>(from < n ? from : n);
    }
  };
  auto stage_ptr = [&](int s) { return s_raw + s * P::kStageBytes; };
  auto load = [&](int s, int row, int rows) {
    uint8_t* st = stage_ptr(s);
    for (int i = threadIdx.x; i < kGradTokens * (kGradCols / 8); i += 256) {
      const int t = i / (kGradCols / 8), c = i % (kGradCols / 8) * 8;
      const bool live = t < rows && col0 + c < a.K;
      cp_async16(smem_u32(st + t * kGradRow + c * 2),
                 live ? a.q + (row + t) * a.q_stride + col0 + c : a.q, live);
    }
    uint8_t* sp = st + kGradTokens * kGradRow;
    for (int i = threadIdx.x; i < kGradTokens * 4 * MB; i += 256) {
      const int t = i / (4 * MB), m = i % (4 * MB) * 4;
      const bool live = t < rows && m < a.r;
      cp_async16(smem_u32(sp + t * P::kPRow + m * 4),
                 live ? a.p + static_cast<int64_t>(row + t) * a.r + m : a.p, live);
    }
  };
  int ahead = 0;  // pieces staged and not yet used
  bool more = count > 0;
  for (int s = 0; s < kGradStages - 1; ++s) {
    int row, rows;
    if (more && (more = next(row, rows))) {
      load(s, row, rows);
      ++ahead;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  int s = 0;
  while (ahead > 0) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kGradStages - 2) : "memory");
    __syncthreads();
    {
      int row, rows;
      if (more && (more = next(row, rows))) {
        load((s + kGradStages - 1) % kGradStages, row, rows);
        ++ahead;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    const uint8_t* st = stage_ptr(s);
    uint8_t* parts = s_raw + kGradStages * P::kStageBytes;
    for (int i = threadIdx.x; i < kGradTokens * 8 * MB; i += 256) {
      const int t = i / (8 * MB), m = i % (8 * MB) * 2;
      float2 f = *reinterpret_cast<const float2*>(st + kGradTokens * kGradRow + t * P::kPRow + m * 4);
#pragma unroll
      for (int h = 0; h < 3; ++h) {
        const uint32_t w = pack_bf16x2(f.x, f.y);
        f.x -= __uint_as_float(w << 16);
        f.y -= __uint_as_float(w & 0xFFFF0000u);
        *reinterpret_cast<uint32_t*>(parts + (h * kGradTokens + t) * P::kSplitRow + m * 2) = w;
      }
    }
    __syncthreads();
    uint32_t bq[kGradTokens / 16][4];  // q: tokens x 16 columns of this warp, transposed on the way
#pragma unroll
    for (int kk = 0; kk < kGradTokens / 16; ++kk)
      ldmatrix_trans(bq[kk], smem_u32(st + (kk * 16 + (lane & 15)) * kGradRow +
                                      (warp * 16 + (lane >> 4) * 8) * 2));
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      float d[2][4] = {};  // this piece's sums
#pragma unroll
      for (int kk = 0; kk < kGradTokens / 16; ++kk)
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          uint32_t w[4];
          const int t = kk * 16 + (lane & 7) + (lane & 16 ? 8 : 0), m = 16 * i + (lane & 8);
          ldmatrix_trans(w, smem_u32(parts + (h * kGradTokens + t) * P::kSplitRow + m * 2));
#pragma unroll
          for (int j = 0; j < 2; ++j)
            mma_16816(d[j], w[0], w[1], w[2], w[3], bq[kk][2 * j], bq[kk][2 * j + 1]);
        }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] += d[j][v];
    }
    --ahead;
    s = (s + 1) % kGradStages;
    __syncthreads();
  }

  float* out = a.out + static_cast<int64_t>(id) * a.r * a.K;
  if (split > 1 && count > 0) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* s_sum = reinterpret_cast<float*>(s_raw);  // [16 MB][128]
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int m = 16 * i + g, c = warp * 16 + 8 * j + 2 * t4;
        *reinterpret_cast<float2*>(s_sum + m * kGradCols + c) = make_float2(acc[i][j][0], acc[i][j][1]);
        *reinterpret_cast<float2*>(s_sum + (m + 8) * kGradCols + c) =
            make_float2(acc[i][j][2], acc[i][j][3]);
      }
    cluster_sync();
    for (int i = rank * 256 + threadIdx.x; i < a.r * kGradCols; i += split * 256) {
      const int m = i / kGradCols, c = i % kGradCols;
      const uint32_t addr = smem_u32(s_sum + i);
      float v = 0.0f;
      for (int o = 0; o < split; ++o) v += ld_cluster(map_to_rank(addr, o));
      if (col0 + c < a.K) {
        float* dst = out + static_cast<int64_t>(m) * a.K + col0 + c;
        *dst = a.accumulate ? *dst + v : v;
      }
    }
    cluster_sync();
    return;
  }
  if (rank > 0 || (count == 0 && a.accumulate)) return;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = 16 * i + g + 8 * h, c = col0 + warp * 16 + 8 * j + 2 * t4;
        if (m < a.r && c < a.K) {
          float2* dst = reinterpret_cast<float2*>(out + static_cast<int64_t>(m) * a.K + c);
          float2 v = make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
          if (a.accumulate) {
            const float2 old = *dst;
            v.x += old.x;
            v.y += old.y;
          }
          *dst = v;
        }
      }
}

// ------------------------------- host side -----------------------------------

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// bf16 [rows, cols] with `stride` values from row to row, boxes of box_rows x 64 values.
// (or fp32, boxes of 32 values)
bool map_2d(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t stride,
            uint32_t box_rows, bool fp32 = false) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {stride * (fp32 ? 4 : 2)};
  const cuuint32_t box[2] = {fp32 ? 32u : 64u, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The library's launch, with clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
void launch_clustered(void (*kern)(KArgs...), dim3 grid, int threads, int smem, int cluster,
                      cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

int pow2_at_most(int64_t v, int most) {
  int p = 1;
  while (2 * p <= v && 2 * p <= most) p *= 2;
  return p;
}

template <int MB, int NB>
moe_status launch_shrink_as(const ShrinkArgs& a, cudaStream_t s) {
  using P = Shrink<MB, NB>;
  auto kern = shrink_kernel<MB, NB>;
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, P::kSmem, mu, done)) return MOE_ERR_CUDA;
  // CTAs a tile for its runs: more than it has runs only costs CTAs that end at once.  The
  // reduction is split over a cluster where the CTAs that have work do not fill the SMs twice.
  const int64_t tiles = ceil_div(a.seg.T, P::kRows), sms = sm_count();
  const int64_t J = std::min<int64_t>(
      {P::kRows, a.seg.n_seg, std::max(ceil_div(2 * static_cast<int64_t>(a.seg.n_seg), tiles), 4 * sms / tiles)});
  const int64_t busy = std::min(tiles * J, tiles + a.seg.n_seg);
  const int split = pow2_at_most(std::min<int64_t>(2 * sms / busy, a.K / 256), 8);
  launch_clustered(kern, dim3(static_cast<unsigned>(tiles * split), static_cast<unsigned>(std::max<int64_t>(J, 1))),
                   32 * kShrinkWarps, P::kSmem, split, s, a, split);
  return launch_status();
}

moe_status launch_shrink(const ShrinkArgs& a, cudaStream_t s) {
  const bool narrow = a.seg.T <= 256;
  const int mb = (a.r + 15) / 16;
  if (mb == 1) return narrow ? launch_shrink_as<1, 1>(a, s) : launch_shrink_as<1, 4>(a, s);
  if (mb == 2) return narrow ? launch_shrink_as<2, 1>(a, s) : launch_shrink_as<2, 4>(a, s);
  if (mb <= 4) return narrow ? launch_shrink_as<4, 1>(a, s) : launch_shrink_as<4, 4>(a, s);
  return narrow ? launch_shrink_as<8, 1>(a, s) : launch_shrink_as<8, 4>(a, s);
}

// bf16 tables [n_adapters, r, cols]: a box that passes r is filled with zeros and not with the
// next adapter's rows.
bool map_tables(CUtensorMap* m, const void* base, uint64_t n_adapters, uint64_t r, uint64_t cols) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {cols, r, n_adapters};
  const cuuint64_t strides[2] = {cols * 2, cols * r * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>((r + 15) / 16 * 16), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operands {
  const void* x;
  int64_t x_stride;
  const void* w;
  const void* table;
};

// Pairs of CTAs that can be resident at once, read once per kernel and device.
template <typename Kernel>
int resident_pairs(Kernel kern, int smem, std::mutex& mu, int (&cache)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sm_count() & ~1));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = sm_count() / 2;
    }
    cache[dev] = n;
  }
  return cache[dev];
}

template <int TN, int S, int CG, bool KMAJ>
moe_status launch_project_as(ProjectArgs a, const Operands& o, cudaStream_t s) {
  using F = Shape<TN, S, CG>;
  auto kern = project_kernel<TN, S, CG, KMAJ>;
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, F::kSmem, mu, done)) return MOE_ERR_CUDA;
  CUtensorMap mw, mx, mt, mu_;
  a.x_rows = static_cast<int>(std::min<int64_t>(TN / CG, ceil_div(a.seg.T, 8) * 8));
  // the weight is [K, N] (rows of N), or for the backward [N, K]
  if (!(KMAJ ? map_2d(&mw, o.w, a.N, a.K, a.K, 128) : map_2d(&mw, o.w, a.K, a.N, a.N, 64)) ||
      !map_2d(&mx, o.x, a.seg.T, a.K, o.x_stride, a.x_rows) ||
      !map_2d(&mu_, a.u, a.seg.T, a.r, a.r, 32, true) || !map_tables(&mt, o.table, a.seg.n_adapters, a.r, a.N))
    return MOE_ERR_CUDA;
  a.n_blocks = static_cast<int>(ceil_div(a.N, 128 * CG));
  a.t_blocks = static_cast<int>(ceil_div(a.seg.T, TN));
  a.slots = std::min(kMaxSlots, F::kTableBytes / (256 * ((a.r + 15) / 16 * 16)));
  a.u_slots = std::min(kMaxSlots, F::kUBytes / ((a.r + 31) / 32 * kUBox));
  // Tokens inner: the weight is read once, the rows stay in the L2.  Rows that outgrow it while
  // the weight does not: columns inner.
  constexpr int64_t kL2Budget = 80ll << 20;
  a.n_inner = static_cast<int64_t>(a.seg.T) * a.K * 2 > kL2Budget &&
              static_cast<int64_t>(a.N) * a.K * 2 <= kL2Budget;
  const int64_t tiles = static_cast<int64_t>(a.n_blocks) * a.t_blocks;
  int64_t clusters = tiles;
  if constexpr (CG == 2) {
    static std::mutex mu2;
    static int pairs[64] = {};
    const int n = resident_pairs(kern, F::kSmem, mu2, pairs);
    if (n <= 0) return MOE_ERR_CUDA;
    clusters = std::min<int64_t>(tiles, n);
  } else if (S == 1) {
    clusters = std::min<int64_t>(tiles, sm_count());
  }
  launch_clustered(kern, dim3(static_cast<unsigned>(clusters * S * CG)), kThreads, F::kSmem, S * CG, s,
                   mw, mx, mt, mu_, a);
  return launch_status();
}

template <bool KMAJ>
moe_status launch_project(const ProjectArgs& a, const Operands& o, cudaStream_t s) {
  const int64_t cols = ceil_div(a.N, 128);
  const int64_t steps = ceil_div(a.K, 64);
  const int64_t sms = sm_count();
  const int T = a.seg.T;
  if (T <= 64) {
    const int split = pow2_at_most(std::min(sms / cols, steps), 8);
    if (split == 8) return launch_project_as<64, 8, 1, KMAJ>(a, o, s);
    if (split == 4) return launch_project_as<64, 4, 1, KMAJ>(a, o, s);
    if (split == 2) return launch_project_as<64, 2, 1, KMAJ>(a, o, s);
    return launch_project_as<64, 1, 1, KMAJ>(a, o, s);
  }
  // Rounds of tiles, in units of a 128 x 128 tile's MMAs a step.
  const int64_t tiles = cols * ceil_div(T, 128);
  const int split = pow2_at_most(std::min(sms / tiles, steps), 8);
  const int64_t flat = split > 1 ? ceil_div(steps, split) : ceil_div(tiles, sms) * steps;
  const int64_t pair = ceil_div(ceil_div(a.N, 256) * ceil_div(T, 256), sms / 2) * steps * 2;
  if (!a.y_fp32 && 10 * pair <= 13 * flat) return launch_project_as<256, 1, 2, KMAJ>(a, o, s);
  if (split == 8) return launch_project_as<128, 8, 1, KMAJ>(a, o, s);
  if (split == 4) return launch_project_as<128, 4, 1, KMAJ>(a, o, s);
  if (split == 2) return launch_project_as<128, 2, 1, KMAJ>(a, o, s);
  return launch_project_as<128, 1, 1, KMAJ>(a, o, s);
}

template <int MB>
moe_status launch_grads_as(const GradArgs& a, cudaStream_t s) {
  using P = Grad<MB>;
  auto kern = grads_kernel<MB>;
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, P::kSmem, mu, done)) return MOE_ERR_CUDA;
  const int64_t blocks = ceil_div(a.K, kGradCols);
  const int64_t active = std::min(a.seg.n_adapters, a.seg.n_seg);
  const int split =
      pow2_at_most(std::min<int64_t>(4 * sm_count() / (blocks * active), a.seg.T / 64), 8);
  launch_clustered(kern, dim3(static_cast<unsigned>(blocks * split), a.seg.n_adapters), 256, P::kSmem,
                   split, s, a, split);
  return launch_status();
}

moe_status launch_grads(const GradArgs& a, cudaStream_t s) {
  const int mb = (a.r + 15) / 16;
  if (mb == 1) return launch_grads_as<1>(a, s);
  if (mb == 2) return launch_grads_as<2>(a, s);
  if (mb <= 4) return launch_grads_as<4>(a, s);
  return launch_grads_as<8>(a, s);
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
}  // namespace moe

using namespace moe;

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
  return launch_project<false>(ProjectArgs{seg, p->d, p->n, p->r, u, y, p->y_stride,
                                           p->y_type == MOE_DTYPE_FP32, 0, 0, 0, 0, 0, 0, dev_status},
                               Operands{x, p->x_stride, w, b}, s);
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
    st = launch_project<true>(ProjectArgs{seg, p->n, p->d, p->r, v, dx, p->d, 0, 0, 0, 0, 0, 0, 0, dev_status},
                              Operands{dy, p->y_stride, w, a}, s);
    if (st != MOE_OK) return st;
  }
  if (da != nullptr) {
    st = launch_grads(GradArgs{seg, p->d, p->r, v, x, p->x_stride, da, accumulate}, s);
    if (st != MOE_OK) return st;
  }
  if (db != nullptr) return launch_grads(GradArgs{seg, p->n, p->r, u, dy, p->y_stride, db, accumulate}, s);
  return MOE_OK;
}
