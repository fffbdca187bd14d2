// Gradient norms over groups of many tensors, and the tensors scaled to a largest norm.
//
//   norm_g = sqrt(sum x^2 over g's tensors),  c_g = min(1, max_norm / (norm_g + 1e-6))
//   (1 where max_norm is infinite)
//   out = round(x c_g)
//
// Bound: HBM (the tensors twice in, once out, less what the second pass finds in the L2).
// The elements of all tensors are one line of chunks (of kChunkBytes, none across two
// tensors), cut into as many equal parts as there are blocks.  Tensors of a group stand
// together, so the pairs (block, group) that occur form a staircase along the line and b + g
// numbers them without gaps or clashes: each block writes the sum of its part of group g to
// partial[b + g], and whoever needs norm g adds the entries of g's blocks, always in the same
// order.  No atomics, no counters: the same bits on every run, and nothing to clear.  The
// second pass walks every part backwards: its end is what the first pass read last.
//
// Squares are summed in fp32 over a thread's share of four chunks (32 fp32 or 64 bf16 values and at most one
// beside them) in chains of eight, so that a sum's path has 12 roundings at most, and in fp64 from there on;
// where those squares leave fp32's range (values beyond 2^60 or below 2^-40) the values are
// scaled by a power of two first, so any finite tensor has its norm.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kBlock = 256;
constexpr int kChunkBytes = 8192;
constexpr int kBatch = 4;  // chunks of one tensor that a block loads at once
constexpr int kVecs = kBatch * kChunkBytes / 16 / kBlock;  // their vectors a thread, at most
constexpr int kPerSm = 2;   // blocks: more of them were slower (four: 617 us for 1.2 GB, two: 554)
constexpr int kMaxBlocks = 1024;

struct ClipArgs {
  const moe_grad_tensor* tensors;
  int n_tensors, n_groups;
  int64_t n_chunks;
  double* partial;  // [gridDim.x + n_groups - 1]
  float max_norm;
  float* norms;
  uint32_t* dev_status;
};

// The last tensor whose first chunk is at or before c: the one that holds it (tensors without
// elements have no chunk and are passed over).  By the whole block, 256 tensors at a time.
__device__ __forceinline__ int tensor_of(const ClipArgs& a, int64_t c) {
  int lo = 0, n = a.n_tensors;
  while (n > 1) {
    const int stride = (n + kBlock - 1) / kBlock;
    const int at = static_cast<int>(threadIdx.x) * stride;
    const int k = __syncthreads_count(at < n && a.tensors[lo + at].first_chunk <= c);
    const int skip = k > 0 ? (k - 1) * stride : 0;
    lo += skip;
    n = min(stride, n - skip);
  }
  return lo;
}

__device__ __forceinline__ int64_t part_begin(int64_t b, int64_t chunks, int64_t parts) {
  return b * chunks / parts;
}
// The part that holds chunk c: the last b with part_begin(b) <= c.
__device__ __forceinline__ int part_of(int64_t c, int64_t chunks, int64_t parts) {
  return static_cast<int>(((c + 1) * parts + chunks - 1) / chunks - 1);
}

__host__ __device__ constexpr int elem_bytes(int type) { return type == MOE_DTYPE_BF16 ? 2 : 4; }
__host__ __device__ constexpr int chunk_elems(int type) { return kChunkBytes / elem_bytes(type); }

__device__ __forceinline__ float value(uint16_t v) { return bf16_bits_to_float(v); }
__device__ __forceinline__ float value(float v) { return v; }

__device__ __forceinline__ void spread(const uint4& v, float (&f)[8]) { unpack8(v, f); }
__device__ __forceinline__ void spread(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}

// This thread's share of up to kBatch chunks of a tensor: of their vectors of 16 bytes (`head`
// elements behind the start, where the source is aligned) and at most one of the elements beside them (fewer than two
// vectors' worth).
struct Share {
  uint4 v[kVecs];
  float edge;
  int edge_at;  // its place, or -1
  int head, vecs;
  void* out;    // of the first chunk
  int type, tensor, group;
  bool in_place;
  __device__ __forceinline__ void load(const moe_grad_tensor& t, int index, int64_t chunk, int chunks) {
    type = t.type;
    tensor = index;
    group = t.group;
    const int size = elem_bytes(type), per = 16 / size;
    const int64_t at = (chunk - t.first_chunk) * chunk_elems(type);
    const int n = static_cast<int>(min(t.count - at, static_cast<int64_t>(chunks) * chunk_elems(type)));
    const uint8_t* src = static_cast<const uint8_t*>(t.grad) + at * size;
    out = static_cast<uint8_t*>(t.out) + at * size;
    in_place = t.grad == t.out;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15u) / size;
    head = min(n, (per - off) % per);
    vecs = (n - head) / per;
    const int tail = n - head - vecs * per;
    const uint4* body = reinterpret_cast<const uint4*>(src + head * size);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int j = i * kBlock + threadIdx.x;
      v[i] = j < vecs ? body[j] : make_uint4(0, 0, 0, 0);
    }
    const int k = threadIdx.x;
    edge_at = k < head ? k : k < head + tail ? vecs * per + k : -1;
    edge = 0.0f;
    if (edge_at >= 0)
      edge = type == MOE_DTYPE_BF16 ? value(reinterpret_cast<const uint16_t*>(src)[edge_at])
                                    : value(reinterpret_cast<const float*>(src)[edge_at]);
  }
  template <int PER>
  __device__ __forceinline__ float sum(float k) const {
    float s[PER];  // a chain for each place in a vector: kVecs additions
#pragma unroll
    for (int e = 0; e < PER; ++e) s[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float f[PER];
      spread(v[i], f);
#pragma unroll
      for (int e = 0; e < PER; ++e) s[e] = fmaf(f[e] * k, f[e] * k, s[e]);
    }
    s[0] = fmaf(edge * k, edge * k, s[0]);
#pragma unroll
    for (int o = PER / 2; o > 0; o /= 2)
#pragma unroll
      for (int e = 0; e < o; ++e) s[e] += s[e + o];
    return s[0];
  }
  template <int PER>
  __device__ __forceinline__ double squares_as() const {
    const float s = sum<PER>(1.0f);
    if (s > 0x1p-80f && s < 0x1p126f) return static_cast<double>(s);
    if (s >= 0x1p126f) return static_cast<double>(sum<PER>(0x1p-75f)) * 0x1p150;
    return static_cast<double>(sum<PER>(0x1p100f)) * 0x1p-200;  // (a NaN stays one)
  }
  __device__ __forceinline__ double squares() const {
    return type == MOE_DTYPE_BF16 ? squares_as<8>() : squares_as<4>();
  }
};

// Sum over the block, the same in every thread.
__device__ __forceinline__ double block_sum(double v, double* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();  // the last sum has been read
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kBlock / 32; ++i) s += s_warp[i];
  return s;
}

__global__ void __launch_bounds__(kBlock, kPerSm) grad_squares_kernel(const ClipArgs a) {
  __shared__ double s_warp[kBlock / 32];
  const int64_t c0 = part_begin(blockIdx.x, a.n_chunks, gridDim.x);
  const int64_t c1 = part_begin(blockIdx.x + 1, a.n_chunks, gridDim.x);
  pdl_wait();
  pdl_trigger();  // the grid is resident as a whole
  for (int g = blockIdx.x * kBlock + threadIdx.x; g < a.n_groups; g += gridDim.x * kBlock)
    a.norms[g] = 0.0f;  // of a group without elements; the others are written by the second pass
  double sum = 0.0;
  int ti = tensor_of(a, c0);
  moe_grad_tensor t = a.tensors[ti];
  auto end_of = [&]() { return t.first_chunk + (t.count + chunk_elems(t.type) - 1) / chunk_elems(t.type); };
  int64_t end = end_of();
  auto fetch = [&](Share& s, int64_t c) {
    while (end <= c) {
      t = a.tensors[++ti];
      end = end_of();
    }
    const int n = static_cast<int>(min(min(end, c1) - c, static_cast<int64_t>(kBatch)));
    s.load(t, ti, c, n);
    return n;
  };
  int group = t.group;
  for (int64_t c = c0; c < c1;) {
    Share now;
    c += fetch(now, c);
    if (now.group != group) {
      const double s = block_sum(sum, s_warp);
      if (threadIdx.x == 0) a.partial[blockIdx.x + group] = s;
      sum = 0.0;
      group = now.group;
    }
    sum += now.squares();
  }
  const double s = block_sum(sum, s_warp);
  if (threadIdx.x == 0) a.partial[blockIdx.x + group] = s;
}

// Norm of the group of tensor t, by the whole block.
__device__ __forceinline__ float group_norm(const ClipArgs& a, const moe_grad_tensor& t, double* s_warp) {
  double v = 0.0;
  const int b0 = part_of(t.group_begin, a.n_chunks, gridDim.x);
  const int b1 = part_of(t.group_end - 1, a.n_chunks, gridDim.x);
  for (int b = b0 + threadIdx.x; b <= b1; b += kBlock) v += __ldcg(a.partial + b + t.group);
  return static_cast<float>(sqrt(block_sum(v, s_warp)));
}

__device__ __forceinline__ uint4 join(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 join(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <typename T>
__device__ __forceinline__ void scale_share(const Share& s, float k) {
  constexpr int kPer = 16 / sizeof(T);
  T* out = static_cast<T*>(s.out);
  if (s.edge_at >= 0) put(out + s.edge_at, s.edge * k);
  out += s.head;
  const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int j = i * kBlock + threadIdx.x;
    if (j >= s.vecs) break;
    float f[kPer];
    spread(s.v[i], f);
#pragma unroll
    for (int e = 0; e < kPer; ++e) f[e] *= k;
    if (aligned) {
      reinterpret_cast<uint4*>(out)[j] = join(f);
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) put(out + j * kPer + e, f[e]);
    }
  }
}

__global__ void __launch_bounds__(kBlock, kPerSm) grad_scale_kernel(const ClipArgs a) {
  __shared__ double s_warp[kBlock / 32];
  const int64_t c0 = part_begin(blockIdx.x, a.n_chunks, gridDim.x);
  const int64_t c1 = part_begin(blockIdx.x + 1, a.n_chunks, gridDim.x);
  // The first pass waited for everything before it and writes only partial and norms: the
  // table and the gradients are read before it has ended.
  int ti = tensor_of(a, c1 - 1);
  moe_grad_tensor t = a.tensors[ti];
  auto fetch = [&](Share& s, int64_t c) {  // chunks up to c
    while (t.count == 0 || t.first_chunk > c) t = a.tensors[--ti];
    const int n = static_cast<int>(min(c + 1 - max(t.first_chunk, c0), static_cast<int64_t>(kBatch)));
    s.load(t, ti, c + 1 - n, n);
    return n;
  };
  int group = -1;
  float k = 1.0f;
  for (int64_t c = c1 - 1; c >= c0;) {
    Share now;
    c -= fetch(now, c);
    if (now.group != group) {
      if (group < 0) pdl_wait();
      group = now.group;
      const moe_grad_tensor& mine = a.tensors[now.tensor];
      const float norm = group_norm(a, mine, s_warp);
      const float q = __fdiv_rn(a.max_norm, norm + 1e-6f);
      // (a NaN stays one; without a limit nothing is scaled, whatever the norm)
      k = q > 1.0f || a.max_norm == __int_as_float(0x7F800000) ? 1.0f : q;
      if (threadIdx.x == 0 && c0 <= mine.group_begin && mine.group_begin < c1) {
        a.norms[group] = norm;
        if (!(norm < __int_as_float(0x7F800000))) report(a.dev_status, MOE_DEV_NONFINITE_INPUT);
      }
    }
    if (k != 1.0f || !now.in_place) {  // (in place, and as it should be: nothing to write)
      if (now.type == MOE_DTYPE_BF16) scale_share<uint16_t>(now, k);
      else scale_share<float>(now, k);
    }
  }
  pdl_trigger();
}

// No elements at all: every norm is zero.
__global__ void __launch_bounds__(kBlock) zero_norms_kernel(int n_groups, float* norms) {
  pdl_wait();
  for (int g = threadIdx.x; g < n_groups; g += kBlock) norms[g] = 0.0f;
  pdl_trigger();
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_grad_plan(int32_t n_tensors, moe_grad_tensor* tensors, int32_t n_groups,
                                 int64_t* n_chunks) {
  if (n_tensors < 0 || n_groups <= 0 || n_chunks == nullptr || (n_tensors > 0 && tensors == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (n_groups > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  int64_t chunks = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    moe_grad_tensor& t = tensors[i];
    if (t.count < 0 || (t.type != MOE_DTYPE_BF16 && t.type != MOE_DTYPE_FP32) || t.group < 0 ||
        t.group >= n_groups || (i > 0 && t.group < tensors[i - 1].group) ||
        (t.count > 0 && (t.grad == nullptr || t.out == nullptr)))
      return MOE_ERR_INVALID_ARG;
    const uintptr_t size = t.type == MOE_DTYPE_BF16 ? 2 : 4;
    if (t.count > 0 && (reinterpret_cast<uintptr_t>(t.grad) % size != 0 ||
                        reinterpret_cast<uintptr_t>(t.out) % size != 0))
      return MOE_ERR_UNSUPPORTED;
    if (t.count > (int64_t(1) << 50)) return MOE_ERR_UNSUPPORTED;
    t.first_chunk = chunks;
    chunks += ceil_div(t.count, chunk_elems(t.type));
    if (chunks > (int64_t(1) << 40)) return MOE_ERR_UNSUPPORTED;
  }
  for (int32_t i = 0; i < n_tensors;) {  // the chunks of each group
    int32_t j = i;
    while (j < n_tensors && tensors[j].group == tensors[i].group) ++j;
    const int64_t end = j < n_tensors ? tensors[j].first_chunk : chunks;
    for (const int64_t begin = tensors[i].first_chunk; i < j; ++i) {
      tensors[i].group_begin = begin;
      tensors[i].group_end = end;
    }
  }
  *n_chunks = chunks;
  return MOE_OK;
}

MOE_API size_t moe_clip_grads_workspace_size(int32_t n_groups) {
  return n_groups <= 0 ? 0 : 8 * (static_cast<size_t>(kMaxBlocks) + n_groups);
}

MOE_API moe_status moe_clip_grads(int32_t n_tensors, const moe_grad_tensor* tensors,
                                  int64_t n_chunks, int32_t n_groups, float max_norm, float* norms,
                                  void* ws, size_t ws_bytes, uint32_t* dev_status,
                                  moe_stream_t stream) {
  if (n_tensors < 0 || n_chunks < 0 || n_groups <= 0 || !(max_norm > 0.0f) || norms == nullptr ||
      (n_chunks > 0 && (n_tensors == 0 || tensors == nullptr || ws == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (n_groups > (1 << 20) || n_chunks > (int64_t(1) << 40) ||
      (reinterpret_cast<uintptr_t>(tensors) & 7u) != 0 || (reinterpret_cast<uintptr_t>(ws) & 7u) != 0 ||
      (reinterpret_cast<uintptr_t>(norms) & 3u) != 0)
    return MOE_ERR_UNSUPPORTED;
  const cudaStream_t s = as_cuda(stream);
  if (n_chunks == 0) {
    launch(zero_norms_kernel, dim3(1), dim3(kBlock), 0, s, n_groups, norms);
    return launch_status();
  }
  if (ws_bytes < moe_clip_grads_workspace_size(n_groups)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const ClipArgs a{tensors, n_tensors, n_groups, n_chunks, static_cast<double*>(ws), max_norm, norms,
                   dev_status};
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(n_chunks, std::min<int64_t>(kPerSm * sm_count(), kMaxBlocks)));
  launch(grad_squares_kernel, dim3(grid), dim3(kBlock), 0, s, a);
  launch(grad_scale_kernel, dim3(grid), dim3(kBlock), 0, s, a);
  return launch_status();
}
