// What the kernels of the projection with adapters share: the segments of rows and their
// adapters, the small tensor-core wrappers, and the projection's launch.
#pragma once

#include <algorithm>

#include "smem.cuh"
#include "umma.cuh"

namespace moe {
namespace adapter {

struct Segments {
  const int32_t* offsets;  // [n_seg + 1], or nullptr: one segment of all rows
  const int32_t* adapter;  // [n_seg]
  int n_seg, T, n_adapters;
};

struct ProjectArgs {
  Segments seg;
  int K, N, r;
  const float* u;         // [T, r]
  const uint16_t* table;  // [n_adapters, r, N]
  void* y;
  int64_t y_stride;
  int y_fp32;
  int n_blocks, t_blocks, n_inner;
  int x_rows;  // rows of a box of x: those behind the batch's last are never staged
  uint32_t* dev_status;
};

struct Operands {
  const void* x;
  int64_t x_stride;
  const void* w;
};

// The projection's shapes (adapter_project.cuh), one translation unit each: `split` CTAs share a
// tile's reduction.  kmaj: the weight's rows are the outputs (the backward).
moe_status project_flat64(const ProjectArgs& a, const Operands& o, int split, cudaStream_t s);
moe_status project_flat64_kmaj(const ProjectArgs& a, const Operands& o, int split, cudaStream_t s);
moe_status project_flat128(const ProjectArgs& a, const Operands& o, int split, cudaStream_t s);
moe_status project_flat128_kmaj(const ProjectArgs& a, const Operands& o, int split, cudaStream_t s);
moe_status project_pair(const ProjectArgs& a, const Operands& o, bool kmaj, cudaStream_t s);

// u [T, r] = scale (x table^T) of each row's own table.
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

// out[e, m, k] = (or +=) sum over e's tokens of p[t, m] q[t, k], of up to two pairs of p and q
// (adapter_grads.cu).
struct GradSide {
  int K;              // 0: left out
  const float* p;     // [T, r]
  const uint16_t* q;  // [T, K]
  int64_t q_stride;
  float* out;         // [n_adapters, r, K]
};
struct GradArgs {
  Segments seg;
  int r;
  GradSide side[2];
  int accumulate;
  int check;  // look the segment table over: no kernel before this one has
  uint32_t* dev_status;
};

moe_status table_grads(const GradArgs& a, cudaStream_t s);

// Segments long enough for tiles of 128 rows (adapter_shrink.cu).
moe_status shrink_long(const ShrinkArgs& a, cudaStream_t s);

namespace {

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

// The segment table, looked over once a call.
__device__ __forceinline__ void check_segments(const Segments& s, uint32_t* dev_status) {
  for (int q = threadIdx.x; q < s.n_seg; q += blockDim.x) {
    const int b = seg_begin(s, q), e = seg_begin(s, q + 1);
    if (b < 0 || e < b || e > s.T) report(dev_status, MOE_DEV_BAD_MAP);
    const int id = __ldg(s.adapter + q);
    if (id < kNone || id >= s.n_adapters) report(dev_status, MOE_DEV_BAD_ADAPTER);
  }
}

// Each segment cut into pieces of `size` rows (the last one shorter): piece `index` of them all,
// by the whole block.  There are at most n_seg + T / size (offsets out of order may name more;
// those are left out).
struct Piece {
  int row, rows, adapter;  // rows = 0: there is no such piece
};
template <int THREADS>
__device__ __forceinline__ Piece piece_of(const Segments& s, int index, int size) {
  __shared__ int s_sum[THREADS / 32];
  __shared__ Piece s_piece;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_piece.rows = 0;
  int64_t before = 0;  // pieces of the segments in front of this round's
  for (int q0 = 0; q0 < s.n_seg; q0 += THREADS) {
    const int q = q0 + static_cast<int>(threadIdx.x);
    int b = 0, e = 0;
    if (q < s.n_seg) seg_rows(s, q, b, e);
    const int n = e > b ? (e - b + size - 1) / size : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();  // (the round before has been read)
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t at = before + incl - n, total = before;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) at += s_sum[w];
      total += s_sum[w];
    }
    if (index >= at && index < at + n) {
      const int row = b + static_cast<int>(index - at) * size;
      s_piece = Piece{row, min(size, e - row), seg_adapter(s, q)};
    }
    before = total;
    if (total > index) break;
  }
  __syncthreads();
  return s_piece;
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

__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// The sum of a float at the same place in every CTA of a cluster of `split`, in the order of the
// ranks.  (All loads are on their way before the first is used.)
__device__ __forceinline__ float sum_of_ranks(uint32_t addr, int split) {
  float v[8];
#pragma unroll
  for (int o = 0; o < 8; ++o) v[o] = o < split ? ld_cluster(map_to_rank(addr, o)) : 0.0f;
  float sum = v[0];
#pragma unroll
  for (int o = 1; o < 8; ++o) sum += v[o];
  return sum;
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

// bf16 [rows, cols] with `stride` values from row to row, boxes of box_rows x 64 values.
inline bool map_2d(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t stride,
            uint32_t box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {stride * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 tables [n_adapters, r, cols], boxes of box_rows x 64 values of one adapter: one that passes
// r is filled with zeros and not with the next adapter's rows.
inline bool map_tables(CUtensorMap* m, const void* base, uint64_t n_adapters, uint64_t r, uint64_t cols,
                       uint32_t box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {cols, r, n_adapters};
  const cuuint64_t strides[2] = {cols * 2, cols * r * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int pow2_at_most(int64_t v, int most) {
  int p = 1;
  while (2 * p <= v && 2 * p <= most) p *= 2;
  return p;
}

}  // namespace
}  // namespace adapter
}  // namespace moe
