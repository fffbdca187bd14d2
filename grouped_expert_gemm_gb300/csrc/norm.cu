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
// Bound: HBM.  A row is read once and held in registers (V chunks of 8 values
// per thread, NW warps a row) through both reductions, so x and r are read once
// and every output written once.
#include "common.cuh"

namespace moe {
namespace {

constexpr float kE4M3Max = 448.0f;
constexpr uint32_t kAbsInf = 0x7F800000u;
constexpr int kMaxNormD = 16384;

struct NormArgs {
  int64_t n, x_stride;
  int d;
  int x32, r32;  // fp32 (else bf16) x and residual stream
  int group;     // scale group of q: MOE_SCALE_ROW or MOE_SCALE_BLOCK128
  int G;         // scales per row
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

// 8 consecutive values of a bf16 or fp32 array.  Plain (coherent) loads: a row's
// output may be written over its input.
__device__ __forceinline__ void load8(const void* p, int is32, int64_t at, float f[8]) {
  if (is32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at), f);
  }
}

__device__ __forceinline__ void store8(void* p, int is32, int64_t at, const float f[8]) {
  if (is32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over the NW warps of a row (every thread gets it; fixed order).  `sh` holds
// two alternating sets of NW floats, so one barrier per reduction is enough.
template <int NW>
__device__ __forceinline__ float row_sum(float v, float* sh, int& phase) {
  v = warp_sum(v);
  if constexpr (NW > 1) {
    float* s = sh + phase * NW;
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) v += s[i];
  }
  return v;
}

template <int NW>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float* sh, int& phase) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if constexpr (NW > 1) {
    uint32_t* s = reinterpret_cast<uint32_t*>(sh + phase * NW);
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) v = max(v, s[i]);
  }
  return v;
}

// Largest |v| of 8 values as fp32 bits (integer order; NaN above Inf).
__device__ __forceinline__ uint32_t amax8(const float f[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

__device__ __forceinline__ float scale_of(uint32_t amax) {
  return amax == 0 ? 1.0f : __fdiv_rn(__uint_as_float(amax), kE4M3Max);
}

__device__ __forceinline__ uint2 quant8(const float f[8], float s) {
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[2 * i], s), __fdiv_rn(f[2 * i + 1], s)),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}

// NW warps hold one row (NW > 1: one row per block; NW = 1: a row per warp).
template <int NW, int V>
__global__ void __launch_bounds__(NW == 1 ? 128 : NW * 32)
add_rms_norm_kernel(const NormArgs a) {
  __shared__ float sh[2 * NW];
  pdl_wait();
  const int rows_per_block = NW == 1 ? static_cast<int>(blockDim.x >> 5) : 1;
  const int tid = NW == 1 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int sub = NW == 1 ? static_cast<int>(threadIdx.x >> 5) : 0;
  const int chunks = a.d / 8;
  int phase = 0;
  bool bad = false;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + sub; row < a.n;
       row += static_cast<int64_t>(gridDim.x) * rows_per_block) {
    const int64_t base = row * a.d;
    float h[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NW * 32;
      if (c < chunks) load8(a.x, a.x32, row * a.x_stride + 8 * c, h[i]);
    }
    float ss = 0.0f;
    if (a.res != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * NW * 32;
        if (c < chunks) {
          float r[8];
          load8(a.res, a.r32, base + 8 * c, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h[i][j] += r[j];
            if (!a.r32) h[i][j] = __bfloat162float(__float2bfloat16_rn(h[i][j]));
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NW * 32;
      if (c < chunks) {
        if (a.res_out != nullptr) store8(a.res_out, a.r32, base + 8 * c, h[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];
      }
    }
    ss = row_sum<NW>(ss, sh, phase);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(ss / static_cast<float>(a.d) + a.eps));
    if (a.rstd != nullptr && tid == 0) a.rstd[row] = rstd;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NW * 32;
      if (c < chunks) {
        float w[8];
        ldg8(a.w, 8 * c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * rstd * w[j];
        if (a.y != nullptr) store8(a.y, 0, base + 8 * c, h[i]);
        top = max(top, amax8(h[i]));
      }
    }
    if (a.q == nullptr) continue;
    if (a.group == MOE_SCALE_ROW) {
      top = row_max<NW>(top, sh, phase);
      const float s = scale_of(top);
      if (tid == 0) a.scales[row] = s;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * NW * 32;
        if (c < chunks) *reinterpret_cast<uint2*>(a.q + base + 8 * c) = quant8(h[i], s);
      }
      bad |= top >= kAbsInf;
    } else {
      // 16 consecutive chunks, one group, lie in one half-warp
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * NW * 32;
        uint32_t m = c < chunks ? amax8(h[i]) : 0u;
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (c < chunks) {
          const float s = scale_of(m);
          if ((c & 15) == 0) a.scales[row * a.G + (c >> 4)] = s;
          *reinterpret_cast<uint2*>(a.q + base + 8 * c) = quant8(h[i], s);
          bad |= m >= kAbsInf;
        }
      }
    }
  }
  if (bad) report(a.dev_status, MOE_DEV_NONFINITE_INPUT);
  pdl_trigger();
}

// --------------------------------- backward ---------------------------------

struct NormBwdArgs {
  int64_t n;
  int d;
  int dy32, x32, r32;
  const void* dy;
  const void* h;
  const float* w;
  const float* rstd;
  const void* dh_out;  // gradient that reaches h from its other readers, or nullptr
  void* dx;
  void* dres;
  float* part;         // [gridDim.x, d] partial weight gradients, or nullptr
};

// The rows of a block go through it in order; each thread keeps the weight
// gradient of its own columns in registers and the block writes one partial row.
template <int NW, int V>
__global__ void __launch_bounds__(NW == 1 ? 128 : NW * 32)
rms_norm_backward_kernel(const NormBwdArgs a) {
  __shared__ float sh[2 * NW];
  __shared__ float sh_dw[NW == 1 ? 3 * V * 256 : 1];
  pdl_wait();
  const int rows_per_block = NW == 1 ? static_cast<int>(blockDim.x >> 5) : 1;
  const int tid = NW == 1 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int sub = NW == 1 ? static_cast<int>(threadIdx.x >> 5) : 0;
  const int chunks = a.d / 8;
  int phase = 0;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + sub; row < a.n;
       row += static_cast<int64_t>(gridDim.x) * rows_per_block) {
    const int64_t base = row * a.d;
    const float rstd = __ldg(a.rstd + row);
    float xh[V][8], u[V][8];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NW * 32;
      if (c < chunks) {
        load8(a.h, a.r32, base + 8 * c, xh[i]);
        load8(a.dy, a.dy32, base + 8 * c, u[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NW * 32;
      if (c < chunks) {
        float w[8];
        ldg8(a.w, 8 * c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xh[i][j] *= rstd;
          dw[i][j] += u[i][j] * xh[i][j];
          u[i][j] *= w[j];
          dot += u[i][j] * xh[i][j];
        }
      }
    }
    dot = row_sum<NW>(dot, sh, phase) / static_cast<float>(a.d);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NW * 32;
      if (c < chunks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = rstd * (u[i][j] - xh[i][j] * dot);
        if (a.dh_out != nullptr) {
          float g[8];
          load8(a.dh_out, a.r32, base + 8 * c, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[i][j] += g[j];
        }
        if (a.dx != nullptr) store8(a.dx, a.x32, base + 8 * c, u[i]);
        if (a.dres != nullptr) store8(a.dres, a.r32, base + 8 * c, u[i]);
      }
    }
  }
  if (a.part != nullptr) {
    if constexpr (NW == 1) {  // the block's warps, summed in warp order
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
        const int c = tid + i * NW * 32;
        if (c < chunks)
          store8(a.part, 1, static_cast<int64_t>(blockIdx.x) * a.d + 8 * c, dw[i]);
      }
    }
  }
  pdl_trigger();
}

// dw = column sums of the partial rows, in a fixed order: 8 interleaved groups of
// rows per column, then the groups in order.
__global__ void __launch_bounds__(256)
weight_grad_kernel(int blocks, int d, const float* __restrict__ part, float* __restrict__ dw) {
  __shared__ float sh[8][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (col < d) {
#pragma unroll 4
    for (int b = g; b < blocks; b += 8) s += part[static_cast<int64_t>(b) * d + col];
  }
  sh[g][lane] = s;
  __syncthreads();
  if (g == 0 && col < d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sh[i][lane];
    dw[col] = s;
  }
  pdl_trigger();
}

// --------------------------------- host side --------------------------------

constexpr int64_t kMaxGrid = 1 << 20;

unsigned forward_grid(int64_t n, int rows_per_block) {
  const int64_t b = ceil_div(n, rows_per_block);
  return static_cast<unsigned>(b > kMaxGrid ? kMaxGrid : b);
}

// Blocks of the backward: two per SM; each writes one partial weight gradient.
int backward_blocks(int64_t n, int rows_per_block) {
  const int64_t b = ceil_div(n, rows_per_block), most = 2 * 152;
  return static_cast<int>(b < most ? b : most);
}

// Widths up to 512 values: a row per warp, four to a block; above: a row per
// block of 8 warps.
bool row_per_warp(int d) { return d <= 512; }

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
  if (st != MOE_OK) return st;
  if (residual == nullptr && p->residual_type != p->x_type) return MOE_ERR_INVALID_ARG;
  if (residual != nullptr && residual_out == nullptr) return MOE_ERR_INVALID_ARG;
  if ((q == nullptr) != (scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (y == nullptr && q == nullptr) return MOE_ERR_INVALID_ARG;
  if (p->n == 0) return MOE_OK;
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
  a.x32 = p->x_type == MOE_DTYPE_FP32;
  a.r32 = p->residual_type == MOE_DTYPE_FP32;
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
  cudaStream_t s = as_cuda(stream);
  const int chunks = p->d / 8;
  if (row_per_warp(p->d)) {
    launch(add_rms_norm_kernel<1, 2>, dim3(forward_grid(p->n, 4)), dim3(128), 0, s, a);
  } else {
    const dim3 grid(forward_grid(p->n, 1)), block(256);
    if (chunks <= 256) launch(add_rms_norm_kernel<8, 1>, grid, block, 0, s, a);
    else if (chunks <= 512) launch(add_rms_norm_kernel<8, 2>, grid, block, 0, s, a);
    else if (chunks <= 1024) launch(add_rms_norm_kernel<8, 4>, grid, block, 0, s, a);
    else launch(add_rms_norm_kernel<8, 8>, grid, block, 0, s, a);
  }
  return launch_status();
}

MOE_API size_t moe_add_rms_norm_backward_workspace_size(const moe_norm_params* p) {
  if (check_norm(p) != MOE_OK) return 0;
  return static_cast<size_t>(backward_blocks(p->n, row_per_warp(p->d) ? 4 : 1)) * p->d *
         sizeof(float);
}

MOE_API moe_status moe_add_rms_norm_backward(const moe_norm_params* p, int32_t dy_type,
                                             const void* dy, const void* h, const float* weight,
                                             const float* rstd, const void* dresidual_out,
                                             void* dx, void* dresidual, float* dweight, void* ws,
                                             size_t ws_bytes, moe_stream_t stream) {
  const moe_status st = check_norm(p);
  if (st != MOE_OK) return st;
  if (dy_type != MOE_DTYPE_BF16 && dy_type != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (dx == nullptr && dresidual == nullptr && dweight == nullptr) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = as_cuda(stream);
  if (p->n == 0) {
    if (dweight != nullptr &&
        cudaMemsetAsync(dweight, 0, static_cast<size_t>(p->d) * sizeof(float), s) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
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
  NormBwdArgs a = {};
  a.n = p->n;
  a.d = p->d;
  a.dy32 = dy_type == MOE_DTYPE_FP32;
  a.x32 = p->x_type == MOE_DTYPE_FP32;
  a.r32 = p->residual_type == MOE_DTYPE_FP32;
  a.dy = dy;
  a.h = h;
  a.w = weight;
  a.rstd = rstd;
  a.dh_out = dresidual_out;
  a.dx = dx;
  a.dres = dresidual;
  a.part = dweight != nullptr ? static_cast<float*>(ws) : nullptr;
  const int chunks = p->d / 8;
  const int blocks = backward_blocks(p->n, row_per_warp(p->d) ? 4 : 1);
  if (row_per_warp(p->d)) {
    launch(rms_norm_backward_kernel<1, 2>, dim3(blocks), dim3(128), 0, s, a);
  } else {
    const dim3 grid(blocks), block(256);
    if (chunks <= 256) launch(rms_norm_backward_kernel<8, 1>, grid, block, 0, s, a);
    else if (chunks <= 512) launch(rms_norm_backward_kernel<8, 2>, grid, block, 0, s, a);
    else if (chunks <= 1024) launch(rms_norm_backward_kernel<8, 4>, grid, block, 0, s, a);
    else launch(rms_norm_backward_kernel<8, 8>, grid, block, 0, s, a);
  }
  if (dweight != nullptr)
    launch(weight_grad_kernel, dim3(static_cast<unsigned>(ceil_div(p->d, 32))), dim3(256), 0, s,
           blocks, p->d, static_cast<const float*>(ws), dweight);
  return launch_status();
}
