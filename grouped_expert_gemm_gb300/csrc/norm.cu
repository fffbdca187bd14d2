// Residual addition and root-mean-square norm with the layer's inputs as its
// outputs -- bf16 token rows and/or the E4M3 dispatch payload -- and its backward.
//
//   h = round(x + r),  rstd = (mean h^2 + eps)^-1/2,  v = h rstd w,
//   y = bf16(v),  s_g = fp32(max over group g of |v| / 448) (1 for a zero group),
//   q = E4M3(v / s_g)
// and with u = w dy, xh = h rstd
//   dh = rstd (u - xh mean(u xh)) + dh_out,   dw = sum over rows of dy xh.
//
// h is rounded to the residual stream's type before it is normalised: the next
// layer and the backward read that stored value, so all of them see one h.  The
// codes are taken from the unrounded fp32 v (one rounding, not bf16 then E4M3).
//
// Bound: HBM.  A row is read once and held in registers (V chunks of 8 values per
// thread) through both reductions, so x and r are read once and every output
// written once.  Blocks are persistent; their next rows are on their way into shared
// memory (bulk copies, the forward and wide backward rows) or registers (the backward
// up to 8,192 values).  Forward, 8,192 x 7,168 (of the copy rate 6.7 TB/s): bf16 84 us
// (6.3 TB/s), fp32 residual 125 (6.1), fp32 both 144 (6.1); backward 96 (6.1), 144 (6.5), 174 (6.1).
#include <math.h>

#include <algorithm>

#include "smem.cuh"

namespace moe {
namespace {

constexpr float kE4M3Max = 448.0f;
constexpr uint32_t kAbsInf = 0x7F800000u;
constexpr int kMaxNormD = 16384;
constexpr int kMaxWarps = 32;
// The rings: warps an SM holds (64 registers), its shared memory, what of it a block takes
// beside its rows (at most), rows a row group has on their way (at most).
constexpr int kRingWarps = 32;
constexpr int kSmBytes = 227 * 1024;
constexpr int kBlockBytes = 2048;
constexpr int kMaxDepth = 4;

struct NormArgs {
  int64_t n, x_stride;
  int d;
  int group;     // scale group of q: MOE_SCALE_ROW or MOE_SCALE_BLOCK128
  int G;         // scales per row
  int nw;        // warps per row
  int depth;     // rows of a row group's ring
  int early;     // the grid is resident at once: dependents may launch right after the wait
  float eps;
  const void* x;
  const void* res;   // nullptr: h = x
  const float* w;
  void* res_out;
  uint16_t* y;
  uint8_t* q;
  float* scales;
  float* rstd;
  uint32_t* dev_status;
};

// 8 consecutive values of a bf16 or fp32 array as raw bits.  Plain (coherent) loads:
// a row's output may be written over its input.
template <bool FP32>
struct Raw {
  uint4 v[FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) +
                                                    at * (FP32 ? 4 : 2));
    v[0] = q[0];
    if constexpr (FP32) v[1] = q[1];
  }
  __device__ __forceinline__ void load_shared(const uint8_t* row, int chunk) {
    const uint4* q = reinterpret_cast<const uint4*>(row) + chunk * (FP32 ? 2 : 1);
    v[0] = q[0];
    if constexpr (FP32) v[1] = q[1];
  }
  __device__ __forceinline__ void get(float f[8]) const {
    if constexpr (FP32) {
      f[0] = __uint_as_float(v[0].x); f[1] = __uint_as_float(v[0].y);
      f[2] = __uint_as_float(v[0].z); f[3] = __uint_as_float(v[0].w);
      f[4] = __uint_as_float(v[1].x); f[5] = __uint_as_float(v[1].y);
      f[6] = __uint_as_float(v[1].z); f[7] = __uint_as_float(v[1].w);
    } else {
      unpack8(v[0], f);
    }
  }
};

__device__ __forceinline__ void store8(void* p, int is32, int64_t at, const float f[8]) {
  if (is32) {
    float* q = static_cast<float*>(p) + at;
    if ((reinterpret_cast<uintptr_t>(q) & 31u) == 0) {  // a whole sector per lane
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "f"(f[0]),
                   "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                   : "memory");
    } else {
      reinterpret_cast<float4*>(q)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(q)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
}

__device__ __forceinline__ void ldg8(const float* p, int64_t at, float f[8]) {
  const float4* q = reinterpret_cast<const float4*>(p + at);
  const float4 a = __ldg(q), b = __ldg(q + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Sum over the nw warps of a row (every thread gets it; fixed order).  `sh` holds
// two alternating sets of kMaxWarps values, so one barrier per reduction is enough.
__device__ __forceinline__ float row_sum(float v, int nw, float* sh, int& phase) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (nw > 1) {
    float* s = sh + phase * kMaxWarps;
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < nw ? s[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, int nw, float* sh, int& phase) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if (nw > 1) {
    uint32_t* s = reinterpret_cast<uint32_t*>(sh + phase * kMaxWarps);
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = __reduce_max_sync(0xFFFFFFFFu, lane < nw ? s[lane] : 0u);
  }
  return v;
}

// Largest |v| of 8 values; NaN if one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t amax8(const float f[8]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
  return __float_as_uint(m) & 0x7FFFFFFFu;  // as bits: integer order, NaN above Inf
}

// amax / 448; 1 where that is zero, which it also is for an amax below 2^-141 (codes of
// v / 0 would be infinite or NaN; of v / 1 they are 0).
__device__ __forceinline__ float scale_of(uint32_t amax) {
  const float s = __fdiv_rn(__uint_as_float(amax), kE4M3Max);
  return s == 0.0f ? 1.0f : s;
}

// 8 codes of v / s as v * (1 / s): one reciprocal a group instead of a division a value
// (with the divisions the 7,168-wide case was bound by instructions, 148 us).  Scales
// below the normal range, whose reciprocal could overflow, divide.
__device__ __forceinline__ uint2 quant8(const float f[8], float s) {
  float v[8];
  if (s >= 0x1p-126f) {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f[i] * inv;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(f[i], s);
  }
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}

// A row group's ring in shared memory: slots of one row's operands, filled by one bulk
// copy an operand and counted on the slot's barrier.
struct Ring {
  uint8_t* base;
  uint32_t bars;  // of its slots
  int depth, bytes;
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ const uint8_t* here() const {
    return base + static_cast<size_t>(slot) * bytes;
  }
  // False: the wait gave up (reported where there is a status word), and the row is
  // whatever the slot holds.
  __device__ __forceinline__ bool wait(volatile int* abort_flag, uint32_t* dev_status) const {
    return wait_bounded(bars + 8 * slot, phase, abort_flag, dev_status);
  }
  __device__ __forceinline__ void next() {
    if (++slot == depth) {
      slot = 0;
      phase ^= 1u;
    }
  }
  // After a wait that gave up: copies on their way land before the block leaves.
  __device__ __forceinline__ void drain() {
    for (int i = 0; i < depth; ++i, next()) wait_drain(bars + 8 * slot, phase ^ 1u);
  }
};

__device__ __forceinline__ void init_ring_bars(uint64_t* bars, int n, int* abort_flag) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < n; ++i) mbar_init(smem_u32(bars + i), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

// A row is held by nw warps: with nw = 1 a block's warps take a row each, else the
// whole block takes one.  RING: blocks are persistent and each row group has `depth`
// rows on their way into shared memory, the next one issued as soon as all have taken
// the current row into registers.  (With the next row in registers instead, four chunks a
// thread, 128 registers: 8,192 x 7,168, block codes, bf16 86 us against 84, fp32 residual
// 171 against 125, both fp32 203 against 144, no residual 72 against 62.)
template <int V, bool X32, bool R32, bool RING>
__global__ void __launch_bounds__(1024)
add_rms_norm_kernel(const NormArgs a) {
  __shared__ float sh[2 * kMaxWarps];
  __shared__ __align__(8) uint64_t bars[4 * kMaxDepth];
  __shared__ int s_abort;
  extern __shared__ __align__(128) uint8_t s_rows[];
  volatile int* abort_flag = &s_abort;
  const int nw = a.nw, span = nw * 32;
  const int rows_per_block = nw == 1 ? static_cast<int>(blockDim.x >> 5) : 1;
  const int tid = nw == 1 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int sub = nw == 1 ? static_cast<int>(threadIdx.x >> 5) : 0;
  if constexpr (RING) init_ring_bars(bars, rows_per_block * a.depth, &s_abort);
  pdl_wait_then_trigger(a.early);
  const int chunks = a.d / 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_block;
  const int x_bytes = a.d * (X32 ? 4 : 2), r_bytes = a.res != nullptr ? a.d * (R32 ? 4 : 2) : 0;
  Ring ring = {s_rows + static_cast<size_t>(sub) * a.depth * (x_bytes + r_bytes),
               smem_u32(bars + sub * a.depth), a.depth, x_bytes + r_bytes};
  int phase = 0;
  bool bad = false;
  Raw<X32> nx[RING ? 1 : V];
  Raw<R32> nr[RING ? 1 : V];
  auto issue = [&](int64_t row, int to) {
    const uint32_t bar = ring.bars + 8 * to, dst = smem_u32(ring.base) + to * ring.bytes;
    mbar_arrive_expect_tx(bar, ring.bytes);
    bulk_load(dst, static_cast<const uint8_t*>(a.x) + row * a.x_stride * (X32 ? 4 : 2), x_bytes, bar);
    if (r_bytes != 0)
      bulk_load(dst + x_bytes, static_cast<const uint8_t*>(a.res) + row * r_bytes, r_bytes, bar);
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + sub;
  if (RING && tid == 0)
    for (int i = 0; i < a.depth && row + i * step < a.n; ++i) issue(row + i * step, i);
  for (; row < a.n; row += step) {
    const int64_t base = row * a.d;
    if constexpr (RING) ring.wait(abort_flag, a.dev_status);
    if constexpr (!RING) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * span;
        if (c < chunks) {
          nx[i].load(a.x, row * a.x_stride + 8 * c);
          if (a.res != nullptr) nr[i].load(a.res, base + 8 * c);
        }
      }
    }
    float h[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * span;
      if (c < chunks) {
        if constexpr (RING) nx[0].load_shared(ring.here(), c);
        nx[RING ? 0 : i].get(h[i]);
        if (a.res != nullptr) {
          float r[8];
          if constexpr (RING) nr[0].load_shared(ring.here() + x_bytes, c);
          nr[RING ? 0 : i].get(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += r[j];
        }
        if constexpr (R32) {
          if (a.res_out != nullptr) store8(a.res_out, 1, base + 8 * c, h[i]);
        } else {  // the stored bf16 sum is what is normalised
          const uint4 p = make_uint4(pack_bf16x2(h[i][0], h[i][1]), pack_bf16x2(h[i][2], h[i][3]),
                                     pack_bf16x2(h[i][4], h[i][5]), pack_bf16x2(h[i][6], h[i][7]));
          if (a.res_out != nullptr)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + base + 8 * c) = p;
          unpack8(p, h[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];
      }
    }
    ss = row_sum(ss, nw, sh, phase);  // (every thread has read the slot)
    if constexpr (RING) {
      if (tid == 0 && row + a.depth * step < a.n && !*abort_flag)
        issue(row + a.depth * step, ring.slot);
      ring.next();
    }
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(ss / static_cast<float>(a.d) + a.eps));
    if (a.rstd != nullptr && tid == 0) a.rstd[row] = rstd;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * span;
      uint32_t m = 0;
      if (c < chunks) {
        float w[8];
        ldg8(a.w, 8 * c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * rstd * w[j];
        if (a.y != nullptr) store8(a.y, 0, base + 8 * c, h[i]);
        if (a.q != nullptr) m = amax8(h[i]);
      }
      if (a.q != nullptr && a.group != MOE_SCALE_ROW) {
        // 16 consecutive chunks, one group, lie in one half-warp
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (c < chunks) {
          const float s = scale_of(m);
          if ((c & 15) == 0) a.scales[row * a.G + (c >> 4)] = s;
          *reinterpret_cast<uint2*>(a.q + base + 8 * c) = quant8(h[i], s);
        }
      }
      top = max(top, m);
    }
    if (a.q != nullptr && a.group == MOE_SCALE_ROW) {
      top = row_max(top, nw, sh, phase);
      const float s = scale_of(top);
      if (tid == 0) a.scales[row] = s;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * span;
        if (c < chunks) *reinterpret_cast<uint2*>(a.q + base + 8 * c) = quant8(h[i], s);
      }
    }
    bad |= top >= kAbsInf;
  }
  if (RING && tid == 0 && *abort_flag) ring.drain();
  if (bad) report(a.dev_status, MOE_DEV_NONFINITE_INPUT);
  if (!a.early) pdl_trigger();
}

// --------------------------------- backward ---------------------------------

struct NormBwdArgs {
  int64_t n;
  int d, nw;
  int depth;  // of the ring (wide rows)
  int early;
  int x32;
  const void* dy;
  const void* h;
  const float* w;
  const float* rstd;
  const void* dh_out;  // gradient that reaches h from its other readers, or nullptr
  void* dx;
  void* dres;
  float* part;         // [gridDim.x, d] partial weight gradients, or nullptr
};

// The block's weight gradient as one partial row.
template <int V>
__device__ __forceinline__ void store_partial(const NormBwdArgs& a, float (&dw)[V][8], float* sh_dw,
                                              int rows_per_block, int sub, int tid, int span) {
  if (a.nw == 1) {  // the block's four warps, summed in warp order
    if (sub > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sh_dw[((sub - 1) * V + i) * 256 + j * 32 + tid] = dw[i][j];
    }
    __syncthreads();
    if (sub == 0) {
      for (int s = 0; s < rows_per_block - 1; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) dw[i][j] += sh_dw[(s * V + i) * 256 + j * 32 + tid];
    }
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * span;
      if (c < a.d / 8) store8(a.part, 1, static_cast<int64_t>(blockIdx.x) * a.d + 8 * c, dw[i]);
    }
  }
}

// The rows of a block go through it in order; each thread keeps the weight
// gradient of its own columns in registers and the block writes one partial row.  The
// next row's values wait in registers (by way of a ring, as in the forward: 8,192 x 7,168
// bf16 104 us against 97, its second pass over the slot's values).
template <bool DY32, bool R32>
__global__ void __launch_bounds__(512)
rms_norm_backward_kernel(const NormBwdArgs a) {
  constexpr int V = 2;
  __shared__ float sh[2 * kMaxWarps];
  __shared__ float sh_dw[3 * V * 256];  // (a row per warp: the other three warps' sums)
  pdl_wait_then_trigger(a.early);
  const int nw = a.nw, span = nw * 32;
  const int rows_per_block = nw == 1 ? static_cast<int>(blockDim.x >> 5) : 1;
  const int tid = nw == 1 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int sub = nw == 1 ? static_cast<int>(threadIdx.x >> 5) : 0;
  const int chunks = a.d / 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_block;
  int phase = 0;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  Raw<R32> nh[V], ng[V];
  Raw<DY32> ndy[V];
  float nrstd = 0.0f;
  auto fetch = [&](int64_t row) {
    nrstd = __ldg(a.rstd + row);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * span;
      if (c < chunks) {
        nh[i].load(a.h, row * a.d + 8 * c);
        ndy[i].load(a.dy, row * a.d + 8 * c);
        if (a.dh_out != nullptr) ng[i].load(a.dh_out, row * a.d + 8 * c);
      }
    }
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + sub;
  if (row < a.n) fetch(row);
  for (; row < a.n; row += step) {
    const int64_t base = row * a.d;
    const float rstd = nrstd;
    float xh[V][8], u[V][8];
    Raw<R32> g[V];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * span;
      if (c < chunks) {
        float w[8];
        ldg8(a.w, 8 * c, w);
        nh[i].get(xh[i]);
        ndy[i].get(u[i]);
        g[i] = ng[i];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xh[i][j] *= rstd;
          dw[i][j] += u[i][j] * xh[i][j];
          u[i][j] *= w[j];
          dot += u[i][j] * xh[i][j];
        }
      }
    }
    if (row + step < a.n) fetch(row + step);
    dot = row_sum(dot, nw, sh, phase) / static_cast<float>(a.d);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * span;
      if (c < chunks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = rstd * (u[i][j] - xh[i][j] * dot);
        if (a.dh_out != nullptr) {
          float f[8];
          g[i].get(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[i][j] += f[j];
        }
        if (a.dx != nullptr) store8(a.dx, a.x32, base + 8 * c, u[i]);
        if (a.dres != nullptr) store8(a.dres, R32, base + 8 * c, u[i]);
      }
    }
  }
  if (a.part != nullptr) store_partial<2>(a, dw, sh_dw, rows_per_block, sub, tid, span);
  if (!a.early) pdl_trigger();
}

// Rows above 8,192 values, whose threads have no registers for the next row: a ring as in
// the forward.  A row's h, dy and dh_out stay in its slot through both phases, so the slot
// is refilled behind the next row's reduction.  4,096 x 12,288 bf16: 93 us; without a
// next row on its way 173.
template <bool DY32, bool R32>
__global__ void __launch_bounds__(1024)
rms_norm_backward_wide_kernel(const NormBwdArgs a) {
  __shared__ float sh[2 * kMaxWarps];
  __shared__ __align__(8) uint64_t bars[kMaxDepth];
  __shared__ int s_abort;
  extern __shared__ __align__(128) uint8_t s_rows[];
  volatile int* abort_flag = &s_abort;
  constexpr int V = 2;
  const int nw = a.nw, span = nw * 32, tid = static_cast<int>(threadIdx.x);
  init_ring_bars(bars, a.depth, &s_abort);
  pdl_wait_then_trigger(a.early);
  const int chunks = a.d / 8;
  const int64_t step = gridDim.x;
  const int h_bytes = a.d * (R32 ? 4 : 2), dy_bytes = a.d * (DY32 ? 4 : 2);
  const int g_bytes = a.dh_out != nullptr ? h_bytes : 0;
  Ring ring = {s_rows, smem_u32(bars), a.depth, h_bytes + dy_bytes + g_bytes};
  auto issue = [&](int64_t row, int to) {
    const uint32_t bar = ring.bars + 8 * to, dst = smem_u32(ring.base) + to * ring.bytes;
    mbar_arrive_expect_tx(bar, ring.bytes);
    bulk_load(dst, static_cast<const uint8_t*>(a.h) + row * h_bytes, h_bytes, bar);
    bulk_load(dst + h_bytes, static_cast<const uint8_t*>(a.dy) + row * dy_bytes, dy_bytes, bar);
    if (g_bytes != 0)
      bulk_load(dst + h_bytes + dy_bytes, static_cast<const uint8_t*>(a.dh_out) + row * g_bytes,
                g_bytes, bar);
  };
  int phase = 0;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  const int64_t first = blockIdx.x;
  int64_t row = first;
  if (tid == 0)
    for (int i = 0; i < a.depth && row + i * step < a.n; ++i) issue(row + i * step, i);
  float next_rstd = row < a.n ? __ldg(a.rstd + row) : 0.0f;
  bool read = true;
  for (; row < a.n; row += step) {
    const int64_t base = row * a.d;
    float rstd = next_rstd;
    if (row + step < a.n) next_rstd = __ldg(a.rstd + row + step);
    // the call has no status word: from a wait that gave up on, the block's rows become
    // NaN, and with them its weight gradient (a slot that is not refilled any more looks
    // full every other time round, so later waits are not asked)
    read = read && ring.wait(abort_flag, nullptr);
    if (!read) rstd = NAN;
    const uint8_t* here = ring.here();
    Raw<R32> h;
    Raw<DY32> dy;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * span;
      if (c < chunks) {
        float w[8], xh[8], u[8];
        ldg8(a.w, 8 * c, w);
        h.load_shared(here, c);
        h.get(xh);
        dy.load_shared(here + h_bytes, c);
        dy.get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xh[j] *= rstd;
          dw[i][j] += u[j] * xh[j];
          dot += u[j] * w[j] * xh[j];
        }
      }
    }
    dot = row_sum(dot, nw, sh, phase) / static_cast<float>(a.d);
    // all are past the row before: its slot takes the row a ring further
    if (tid == 0 && a.depth > 1 && row != first && row + (a.depth - 1) * step < a.n && !*abort_flag)
      issue(row + (a.depth - 1) * step, ring.slot == 0 ? a.depth - 1 : ring.slot - 1);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * span;
      if (c < chunks) {
        float w[8], xh[8], u[8];
        ldg8(a.w, 8 * c, w);
        h.load_shared(here, c);
        h.get(xh);
        dy.load_shared(here + h_bytes, c);
        dy.get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = rstd * (u[j] * w[j] - xh[j] * rstd * dot);
        if (a.dh_out != nullptr) {
          float f[8];
          h.load_shared(here + h_bytes + dy_bytes, c);
          h.get(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] += f[j];
        }
        if (a.dx != nullptr) store8(a.dx, a.x32, base + 8 * c, u);
        if (a.dres != nullptr) store8(a.dres, R32, base + 8 * c, u);
      }
    }
    if (a.depth == 1) {  // (rows of which two do not fit)
      __syncthreads();
      if (tid == 0 && row + step < a.n && !*abort_flag) issue(row + step, 0);
    }
    ring.next();
  }
  if (tid == 0 && *abort_flag) ring.drain();
  if (a.part != nullptr) store_partial<V>(a, dw, nullptr, 1, 0, tid, span);
  if (!a.early) pdl_trigger();
}

// dw = column sums of the partial rows, in a fixed order: 32 interleaved groups of
// rows per column, then the groups in order.
__global__ void __launch_bounds__(1024)
weight_grad_kernel(int blocks, int d, const float* __restrict__ part, float* __restrict__ dw,
                   int early) {
  __shared__ float sh[32][33];
  pdl_wait_then_trigger(early);
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (col < d) {
#pragma unroll 10
    for (int b = g; b < blocks; b += 32) s += part[static_cast<int64_t>(b) * d + col];
  }
  sh[g][lane] = s;
  __syncthreads();
  // warp g adds column g's 32 group sums
  s = sh[lane][g];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane == 0 && blockIdx.x * 32 + g < d) dw[blockIdx.x * 32 + g] = s;
  if (!early) pdl_trigger();
}

// --------------------------------- host side --------------------------------

// How a pass lays its rows out: V chunks of 8 values per thread, nw warps a row
// (one: four rows to a block), and for the ring persistent blocks.
struct Plan {
  int V, nw, threads, blocks;
  int depth = 0, smem = 0;  // of the ring
};

// Two chunks a thread (four: 86.6 us at 8,192 x 7,168 bf16, fewer warps to hide the
// reductions).  As many blocks on an SM as its warps and shared memory hold with one row
// each on its way (its copy then runs behind the second half of the row before); only
// where a block has an SM to itself, rows above 8,192 values, does it take more (4,096 x
// 12,288 bf16 forward 75 us, with one 79).  With more everywhere the forward alone is the
// same, but 4,096 x 4,096 forward and backward in turn took 63 to 72 us against 62.
Plan plan_ring(int64_t n, int d, int row_bytes) {
  Plan p;
  p.V = 2;
  p.nw = static_cast<int>(ceil_div(d / 8, 64));
  const int groups = p.nw == 1 ? 4 : 1, rows = groups * row_bytes;
  p.threads = 32 * groups * p.nw;
  int per_sm = kRingWarps / (p.threads / 32);
  while (per_sm > 1 && per_sm * (rows + kBlockBytes) > kSmBytes) --per_sm;
  p.depth = per_sm > 1 ? 1 : std::min(kMaxDepth, (kSmBytes - kBlockBytes) / rows);
  p.smem = p.depth * rows;
  p.blocks = static_cast<int>(
      std::min<int64_t>(ceil_div(n, groups), static_cast<int64_t>(sm_count()) * per_sm));
  return p;
}

// Forward: rows fewer than the SMs are latency-bound and take one chunk a thread straight
// from global memory.
Plan plan_forward(int64_t n, int d, int row_bytes) {
  if (n > sm_count() || d > 8192) return plan_ring(n, d, row_bytes);
  Plan p;
  p.V = 1;
  p.nw = static_cast<int>(ceil_div(d / 8, 32));
  p.threads = 32 * (p.nw == 1 ? 4 : p.nw);
  p.blocks = static_cast<int>(ceil_div(n, p.nw == 1 ? 4 : 1));
  return p;
}

// Backward: two chunks a thread, each block writes one partial row of the weight
// gradient.  Wide rows count as if dh_out were given, so that the order of the sums does
// not depend on it.
Plan plan_backward(int64_t n, int d, bool dy32, bool r32) {
  if (d > 8192) return plan_ring(n, d, d * ((dy32 ? 4 : 2) + (r32 ? 8 : 4)));
  Plan p;
  p.V = 2;
  p.nw = static_cast<int>(ceil_div(d / 8, 64));
  const int warps = p.nw == 1 ? 4 : p.nw;
  p.threads = 32 * warps;
  const int per_sm = std::max(1, 16 / warps);
  p.blocks = static_cast<int>(std::min<int64_t>(ceil_div(n, p.nw == 1 ? 4 : 1),
                                                static_cast<int64_t>(sm_count()) * per_sm));
  return p;
}

template <int V, bool X32, bool R32, bool RING>
bool launch_forward_as(const NormArgs& a, const Plan& p, cudaStream_t s) {
  auto kern = add_rms_norm_kernel<V, X32, R32, RING>;
  if constexpr (RING) {
    static std::mutex mu;
    static bool done[64] = {};
    if (!opt_in(kern, kSmBytes - kBlockBytes, mu, done)) return false;
  }
  launch(kern, dim3(p.blocks), dim3(p.threads), p.smem, s, a);
  return true;
}

template <int V, bool RING>
bool launch_forward(const NormArgs& a, bool x32, bool r32, const Plan& p, cudaStream_t s) {
  if (x32)
    return r32 ? launch_forward_as<V, true, true, RING>(a, p, s)
               : launch_forward_as<V, true, false, RING>(a, p, s);
  return r32 ? launch_forward_as<V, false, true, RING>(a, p, s)
             : launch_forward_as<V, false, false, RING>(a, p, s);
}

template <bool DY32, bool R32>
bool launch_backward(const NormBwdArgs& a, const Plan& p, cudaStream_t s) {
  if (p.depth == 0) {
    launch(rms_norm_backward_kernel<DY32, R32>, dim3(p.blocks), dim3(p.threads), 0, s, a);
    return true;
  }
  auto kern = rms_norm_backward_wide_kernel<DY32, R32>;
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, kSmBytes - kBlockBytes, mu, done)) return false;
  launch(kern, dim3(p.blocks), dim3(p.threads), p.smem, s, a);
  return true;
}

moe_status check_norm(const moe_norm_params* p) {
  if (p == nullptr || p->n < 0 || p->d <= 0) return MOE_ERR_INVALID_ARG;
  if (p->x_type != MOE_DTYPE_BF16 && p->x_type != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (p->residual_type != MOE_DTYPE_BF16 && p->residual_type != MOE_DTYPE_FP32)
    return MOE_ERR_INVALID_ARG;
  if (p->group != MOE_SCALE_ROW && p->group != MOE_SCALE_BLOCK128) return MOE_ERR_INVALID_ARG;
  if (!(p->eps > 0.0f) || !(p->eps < 1e30f)) return MOE_ERR_INVALID_ARG;
  if (p->x_stride < p->d) return MOE_ERR_INVALID_ARG;
  if (p->d % 8 != 0 || p->d > kMaxNormD || p->x_stride % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (p->n > (int64_t(1) << 40) / p->d || p->x_stride > (int64_t(1) << 40) / (p->n + 1))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_add_rms_norm(const moe_norm_params* p, const void* x, const void* residual,
                                    const float* weight, void* residual_out, moe_bf16* y,
                                    moe_fp8* q, float* scales, float* rstd, uint32_t* dev_status,
                                    moe_stream_t stream) {
  const moe_status st = check_norm(p);
  if (st != MOE_OK || p->n == 0) return st;
  if (residual == nullptr && p->residual_type != p->x_type) return MOE_ERR_INVALID_ARG;
  if (residual != nullptr && residual_out == nullptr) return MOE_ERR_INVALID_ARG;
  if ((q == nullptr) != (scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (y == nullptr && q == nullptr) return MOE_ERR_INVALID_ARG;
  if (x == nullptr || weight == nullptr) return MOE_ERR_INVALID_ARG;
  if (q != nullptr && p->d % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) ||
      !aligned16(y) || !aligned16(q) || (reinterpret_cast<uintptr_t>(scales) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0)
    return MOE_ERR_UNSUPPORTED;
  NormArgs a = {};
  a.n = p->n;
  a.x_stride = p->x_stride;
  a.d = p->d;
  a.group = p->group;
  a.G = p->group == MOE_SCALE_ROW ? 1 : static_cast<int>(ceil_div(p->d, 128));
  a.eps = p->eps;
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.res_out = residual_out;
  a.y = y;
  a.q = q;
  a.scales = scales;
  a.rstd = rstd;
  a.dev_status = dev_status;
  const bool x32 = p->x_type == MOE_DTYPE_FP32, r32 = p->residual_type == MOE_DTYPE_FP32;
  const Plan pl =
      plan_forward(p->n, p->d, p->d * ((x32 ? 4 : 2) + (residual == nullptr ? 0 : r32 ? 4 : 2)));
  a.nw = pl.nw;
  a.depth = pl.depth;
  a.early = one_wave(pl.blocks);
  const cudaStream_t s = as_cuda(stream);
  const bool ok = pl.V == 1 ? launch_forward<1, false>(a, x32, r32, pl, s)
                            : launch_forward<2, true>(a, x32, r32, pl, s);
  return ok ? launch_status() : MOE_ERR_CUDA;
}

MOE_API size_t moe_add_rms_norm_backward_workspace_size(const moe_norm_params* p) {
  if (check_norm(p) != MOE_OK) return 0;
  // (of the two types of dy the narrower one has more blocks)
  const int blocks = plan_backward(p->n, p->d, false, p->residual_type == MOE_DTYPE_FP32).blocks;
  return static_cast<size_t>(blocks) * p->d * sizeof(float);
}

MOE_API moe_status moe_add_rms_norm_backward(const moe_norm_params* p, int32_t dy_type,
                                             const void* dy, const void* h, const float* weight,
                                             const float* rstd, const void* dresidual_out,
                                             void* dx, void* dresidual, float* dweight, void* ws,
                                             size_t ws_bytes, moe_stream_t stream) {
  const moe_status st = check_norm(p);
  if (st != MOE_OK) return st;
  if (dy_type != MOE_DTYPE_BF16 && dy_type != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = as_cuda(stream);
  if (p->n == 0) {  // (empty tensors have no address)
    if (dweight != nullptr &&
        cudaMemsetAsync(dweight, 0, static_cast<size_t>(p->d) * sizeof(float), s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (dx == nullptr && dresidual == nullptr && dweight == nullptr) return MOE_ERR_INVALID_ARG;
  if (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(dresidual_out) ||
      !aligned16(dx) || !aligned16(dresidual) || !aligned16(ws) ||
      (reinterpret_cast<uintptr_t>(rstd) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(dweight) & 3u) != 0)
    return MOE_ERR_UNSUPPORTED;
  if (dweight != nullptr) {
    if (ws == nullptr) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_add_rms_norm_backward_workspace_size(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  const bool r32 = p->residual_type == MOE_DTYPE_FP32, dy32 = dy_type == MOE_DTYPE_FP32;
  const Plan pl = plan_backward(p->n, p->d, dy32, r32);
  NormBwdArgs a = {};
  a.n = p->n;
  a.d = p->d;
  a.nw = pl.nw;
  a.depth = pl.depth;
  a.early = one_wave(pl.blocks);
  a.x32 = p->x_type == MOE_DTYPE_FP32;
  a.dy = dy;
  a.h = h;
  a.w = weight;
  a.rstd = rstd;
  a.dh_out = dresidual_out;
  a.dx = dx;
  a.dres = dresidual;
  a.part = dweight != nullptr ? static_cast<float*>(ws) : nullptr;
  const bool ok = dy32 ? (r32 ? launch_backward<true, true>(a, pl, s) : launch_backward<true, false>(a, pl, s))
                       : (r32 ? launch_backward<false, true>(a, pl, s) : launch_backward<false, false>(a, pl, s));
  if (!ok) return MOE_ERR_CUDA;
  if (dweight != nullptr)
    launch(weight_grad_kernel, dim3(static_cast<unsigned>(ceil_div(p->d, 32))), dim3(1024), 0, s,
           pl.blocks, p->d, static_cast<const float*>(ws), dweight,
           static_cast<int>(one_wave(ceil_div(p->d, 32))));
  return launch_status();
}
