// Grouped SwiGLU product over ragged row segments with E4M3 rows, weights and
// intermediate on the 5th-generation tensor cores (tcgen05.mma kind::f8f6f4).
//
//   X = xq * xs[row, k / 128],  W = wq * ws[n / 128, k / 128]
//   G = X Wg^T, U = X Wu^T;  H = SiLU(G) U, hq = E4M3(H / hs), hs = amax / 448 of the
//   row's 128 columns;  y = bf16((hq hs) Wd^T)
// (weights stored [N, K], K contiguous: both operands are K-major).
//
// Bound: decode sizes HBM (the touched experts' weights), 94 us for the 115 to 120 touched
// experts of a 2048 x 768 decode bucket (562 MB, 6.0 TB/s, 89 % of the copy rate).  Large
// segments: the MMAs.  A product without the per-block sums takes 735 cycles a block and CTA
// (3.07 PFLOP/s); the down pass of 8 x 1024 rows, 14336 x 4096, takes 895 (2.4 to 2.5 PFLOP/s),
// gate/up with its SwiGLU and codes 984 (2.3).  Clock stamps there: the promotion warps
// wait 170 to 215 cycles a block for its sums and hand its buffer back 400 to 455 after they
// came, well before the other buffer's MMAs end; the issuer waits 150 for a buffer and 85
// for operands.  Why the MMAs are slower beside the reads is not shown (the port of the
// tensor memory was busy a third of the time).
//
// One reduction block of 128 is one pipeline stage, one row of the 128-byte
// swizzle and one scale block.  The tensor core sums the block's codes into a
// tensor-memory buffer of its own; the promotion warps read it, multiply by the
// row's and the weight block's scales and add in fp32 registers:
//   acc[m, n] += part[m, n] * (xs[m, kb] * ws[n / 128, kb]).
// The scales are arbitrary fp32 values, so they cannot ride in the MMA's own
// power-of-two scale factors.
//
// Tile: 128 rows x 256 weight columns (gate/up: 128 gate + the same 128 up, so a
// tile makes one whole scale group of H; down: 256 columns of y).  Roles of the 320
// threads, one CTA per SM, persistent over the tiles:
//   warp 0       TMA producer: [128 x 128] codes of A, two [128 x 128] of B, 48 KB
//                a stage, four stages
//   warp 1       allocates tensor memory; lane 0 issues four MMAs (K = 32) a stage
//   warps 2..9   promotion and epilogue: warp w reads lanes 32 (w % 4).., columns of
//                half (w - 2) / 4; 128 fp32 sums per thread
// Two tensor-memory buffers of 256 columns: block kb + 1 is summed while kb is
// promoted.  With few tiles and a long reduction a cluster of two or four CTAs takes each
// tile, a part of the blocks to a CTA; every CTA then sends its sums of the other CTAs'
// rows to them through distributed shared memory and finishes its own quarter or half
// (two rounds of a tree, with rank 0 alone in the epilogue, took 2 us longer a pass).
// Every wait is bounded (MOE_DEV_TIMEOUT), as in the bf16 pass.
#include <algorithm>

#include "smem.cuh"
#include "umma.cuh"

namespace moe {
namespace {

constexpr int kMaxSeg = 1024;
constexpr int kBM = 128;                   // rows per tile
constexpr int kBK = 128;                   // codes per stage and scale block
constexpr int kABytes = kBM * kBK;         // 16 KB
constexpr int kBBox = 128 * kBK;           // 16 KB: one box of 128 weight rows
constexpr int kStageBytes = kABytes + 2 * kBBox;
constexpr int kStages = 4;
constexpr int kAccCols = 256;
constexpr int kThreads = 320;
constexpr int kBars = 2 * kStages + 14;  // (an even number)
constexpr int kWarpSums = 32 * 128 * 4;  // a promotion warp's sums, in bytes

constexpr float kE4M3Max = 448.0f;
constexpr uint32_t kAbsInf = 0x7F800000u;

struct W8Args {
  const int32_t* seg_begin;
  const int32_t* seg_count;
  int n_seg, K, N, max_rows;
  int GK, GN;          // scale blocks along K and N
  const float* as;     // [max_rows, GK]
  const float* bs0;    // [n_seg, GN, GK]: gate, or down
  const float* bs1;    // up
  uint8_t* hq;         // gate/up
  float* hs;           // [max_rows, GN]
  uint16_t* y;         // down
  uint32_t* dev_status;
  int m_outer;
  int chained;         // few-rows down pass right behind its gate/up pass
};

struct Tile {
  int seg, row0, rows, nb;
};

struct Table {
  volatile int* abort_flag;
  uint32_t* tmem_slot;
  int* warp_tot;
  int* start;   // [n_seg + 1] first tile of a segment
  int* begin;
  int* count;
};
__host__ __device__ constexpr int table_bytes(int n_seg) { return (8 + 3 * n_seg + 8) * 4; }

__device__ __forceinline__ Table carve_table(int* p, int n_seg) {
  Table t;
  t.abort_flag = p;
  t.tmem_slot = reinterpret_cast<uint32_t*>(p + 1);
  t.warp_tot = p + 4;
  t.start = p + 8;
  t.begin = t.start + n_seg + 1;
  t.count = t.begin + n_seg;
  return t;
}

// Tile t: inside a segment n-block outer / m-block inner, or the reverse (m_outer).
__device__ __forceinline__ Tile tile_of(int t, const Table& tb, int n_seg, int bm, int n_blocks,
                                        int m_outer) {
  int lo = 0, hi = n_seg - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tb.start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int local = t - tb.start[lo];
  const int m_blocks = (tb.count[lo] + bm - 1) / bm;
  Tile tl;
  tl.seg = lo;
  tl.nb = m_outer ? local % n_blocks : local / m_blocks;
  const int mb = m_outer ? local / n_blocks : local % m_blocks;
  tl.row0 = tb.begin[lo] + mb * bm;
  tl.rows = min(bm, tb.count[lo] - mb * bm);
  return tl;
}

// Tile counts of segments that overlap (not allowed, but nothing outside the arrays is to be
// touched) may pass 2^31: sums stop there.  Both operands are below 2^31.
__device__ __forceinline__ int add_tiles(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), 0x7FFFFFFFu));
}

// Segment table by 128 threads (tid 0..127 of named barrier 1): segments outside
// the row space are reported and treated as empty, and all of them where they have more
// tiles than numbers (check_shape: not if they are disjoint).
__device__ __forceinline__ void build_table(const W8Args& a, int bm, int n_blocks, int tid,
                                            const Table& tb) {
  const int lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_seg + 127) / 128;
  const int q0 = tid * per, q1 = min(a.n_seg, q0 + per);
  int local = 0;
  for (int q = q0; q < q1; ++q) {
    int b = __ldg(a.seg_begin + q), c = __ldg(a.seg_count + q);
    if (c < 0 || b < 0 || static_cast<int64_t>(b) + c > a.max_rows) {
      if (c != 0) report(a.dev_status, MOE_DEV_BAD_ROW);
      b = 0;
      c = 0;
    }
    tb.begin[q] = b;
    tb.count[q] = c;
    local = add_tiles(local, ((c + bm - 1) / bm) * n_blocks);
  }
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl = add_tiles(incl, v);
  }
  if (lane == 31) tb.warp_tot[warp] = incl;
  asm volatile("bar.sync 1, 128;" ::: "memory");
  int run = incl - local;
  for (int w = 0; w < warp; ++w) run = add_tiles(run, tb.warp_tot[w]);
  for (int q = q0; q < q1; ++q) {
    tb.start[q] = run;
    run = add_tiles(run, ((tb.count[q] + bm - 1) / bm) * n_blocks);
  }
  if (tid == 127) {
    int total = add_tiles(add_tiles(tb.warp_tot[0], tb.warp_tot[1]),
                          add_tiles(tb.warp_tot[2], tb.warp_tot[3]));
    if (total > 0x7FFFFFFF - 0x10000) {  // (and a CTA's next tile's number is one too)
      report(a.dev_status, MOE_DEV_BAD_ROW);
      total = 0;
    }
    tb.start[a.n_seg] = total;
  }
}

// amax / 448; 1 where that is zero, which it also is for an amax below 2^-141 (codes of
// v / 0 would be infinite or NaN; of v / 1 they are 0).
__device__ __forceinline__ float scale_of(uint32_t amax) {
  const float s = __fdiv_rn(__uint_as_float(amax), kE4M3Max);
  return s == 0.0f ? 1.0f : s;
}

// 32 consecutive bytes (aligned to 16): one 32-byte store where the address allows
// it -- a whole sector per lane -- else two of 16.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8]) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    uint4* q = static_cast<uint4*>(dst);
    q[0] = make_uint4(v[0], v[1], v[2], v[3]);
    q[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// acc += part * s on 16 columns.
__device__ __forceinline__ void promote16(const uint32_t (&part)[16], float s, float2* acc) {
  const float2 s2 = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    acc[i] = __ffma2_rn(make_float2(__uint_as_float(part[2 * i]), __uint_as_float(part[2 * i + 1])),
                        s2, acc[i]);
}

template <bool SWIGLU, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
grouped_w8_kernel(const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_b0,
                  const __grid_constant__ CUtensorMap map_b1, const W8Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stage_base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // bars: full[S], empty[S], tfull[2], tempty[2], amax[4], drain, go[4], red
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage_base + kStages * kStageBytes);
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(bars + kBars);  // [2][2][128]
  const Table tb = carve_table(reinterpret_cast<int*>(s_amax + 512), a.n_seg);
  volatile int* abort_flag = tb.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = SPLIT > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / SPLIT, step = static_cast<int>(gridDim.x) / SPLIT;
  const int kb0 = rank * a.GK / SPLIT, kb1 = (rank + 1) * a.GK / SPLIT;
  const int n_blocks = (a.N + (SWIGLU ? 127 : 255)) / (SWIGLU ? 128 : 256);

  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + kStages + s); };
  auto tfull_bar = [&](int b) { return smem_u32(bars + 2 * kStages + b); };
  auto tempty_bar = [&](int b) { return smem_u32(bars + 2 * kStages + 2 + b); };
  auto amax_bar = [&](int q) { return smem_u32(bars + 2 * kStages + 4 + q); };
  const uint32_t drain_bar = smem_u32(bars + 2 * kStages + 8);
  auto go_bar = [&](int i) { return smem_u32(bars + 2 * kStages + 9 + i); };
  const uint32_t red_bar = smem_u32(bars + 2 * kStages + 13);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 8);  // one arrival per promotion warp
    }
    for (int q = 0; q < 4; ++q) mbar_init(amax_bar(q), 2);  // the two warps of a lane quadrant
    mbar_init(drain_bar, 1);
    for (int i = 0; i < 4; ++i) mbar_init(go_bar(i), 1);
    mbar_init(red_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) umma_alloc(smem_u32(tb.tmem_slot), 2 * kAccCols);
  pdl_wait();
  if (threadIdx.x >= 64 && threadIdx.x < 192)
    build_table(a, kBM, n_blocks, threadIdx.x - 64, tb);
  umma_fence_before();
  if constexpr (SPLIT > 1) cluster_sync();  // the partners' barriers are initialised
  else __syncthreads();
  umma_fence_after();
  bool awaited = false;  // the partners' sums
  const uint32_t tmem = *tb.tmem_slot;
  int total = tb.start[a.n_seg];
  if (SPLIT > 1 && total > step) {  // only segments that overlap have more tiles than clusters
    if (threadIdx.x == 0) report(a.dev_status, MOE_DEV_BAD_ROW);
    total = step;
  }

  if (warp < 2) {
    if (warp == 0 && lane == 0) {
      // ---- TMA producer ----
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        const Tile tl = tile_of(t, tb, a.n_seg, kBM, n_blocks, a.m_outer);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bounded(empty_bar(s), ph ^ 1u, abort_flag, a.dev_status)) { ok = false; break; }
          const uint32_t st = smem_u32(stage_base + s * kStageBytes);
          mbar_arrive_expect_tx(full_bar(s), kStageBytes);
          tma_load_2d(st, &map_a, full_bar(s), kb * kBK, tl.row0);
          if (SWIGLU) {
            tma_load_3d(st + kABytes, &map_b0, full_bar(s), kb * kBK, tl.nb * 128, tl.seg);
            tma_load_3d(st + kABytes + kBBox, &map_b1, full_bar(s), kb * kBK, tl.nb * 128, tl.seg);
          } else {
            tma_load_3d(st + kABytes, &map_b0, full_bar(s), kb * kBK, tl.nb * 256, tl.seg);
            tma_load_3d(st + kABytes + kBBox, &map_b0, full_bar(s), kb * kBK, tl.nb * 256 + 128,
                        tl.seg);
          }
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
      if (!ok) {  // copies in flight land before the shared memory is given up
        for (int i = 0; i < kStages; ++i) {
          if (--s < 0) { s = kStages - 1; ph ^= 1u; }
          wait_drain(full_bar(s), ph);
        }
      }
    } else if (warp == 1 && lane == 0) {
      // ---- MMA issuer ----
      constexpr uint32_t idesc = umma_idesc_e4m3(kBM, kAccCols);
      int s = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true, issued = false;
      for (int t = first; t < total && ok; t += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bounded(tempty_bar(buf), acc_ph ^ 1u, abort_flag, a.dev_status) ||
              !wait_bounded(full_bar(s), ph, abort_flag, a.dev_status)) {
            ok = false;
            break;
          }
          umma_fence_after();
          const uint32_t st = smem_u32(stage_base + s * kStageBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f8(tmem + buf * kAccCols, umma_desc(st + kk * 32), umma_desc(st + kABytes + kk * 32),
                    idesc, kk > 0);
          issued = true;
          umma_commit(empty_bar(s));
          umma_commit(tfull_bar(buf));
          if constexpr (SPLIT > 1)
            if (kb + 1 == kb1) umma_commit_multicast(go_bar(rank), (1 << SPLIT) - 1);
          if (++s == kStages) { s = 0; ph ^= 1u; }
          if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
        }
      }
      if (!ok && issued) {
        umma_commit(drain_bar);
        wait_drain(drain_bar, 0);
      }
    }
  } else {
    // ---- promotion and epilogue ----
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int r = quad * 32 + lane;
    const uint32_t taddr0 = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // columns of the two 64-wide pieces this thread sums, and their scale blocks
    const int c0 = SWIGLU ? 64 * half : 128 * half;
    const int c1 = SWIGLU ? 128 + 64 * half : 128 * half + 64;
    int buf = 0, parity = 0;
    uint32_t acc_ph = 0, tile_ph = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const Tile tl = tile_of(t, tb, a.n_seg, kBM, n_blocks, a.m_outer);
      const bool live = r < tl.rows;
      const int64_t row = min(tl.row0 + r, a.max_rows - 1);
      const float* as = a.as + row * a.GK;
      const int nblk = SWIGLU ? tl.nb : min(2 * tl.nb + half, a.GN - 1);
      const int64_t boff = (static_cast<int64_t>(tl.seg) * a.GN + nblk) * a.GK;
      const float* b0 = a.bs0 + boff;
      const float* b1 = SWIGLU ? a.bs1 + boff : b0;
      float2 acc0[32], acc1[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc0[i] = acc1[i] = make_float2(0.0f, 0.0f);
      float sa = __ldg(as + kb0), w0 = __ldg(b0 + kb0), w1 = __ldg(b1 + kb0);
      for (int kb = kb0; kb < kb1; ++kb) {
        const float s0 = sa * w0, s1 = sa * w1;
        if (kb + 1 < kb1) {
          sa = __ldg(as + kb + 1);
          w0 = __ldg(b0 + kb + 1);
          w1 = __ldg(b1 + kb + 1);
        }
        if (!__all_sync(0xFFFFFFFFu,
                        wait_bounded(tfull_bar(buf), acc_ph, abort_flag, a.dev_status))) {
          ok = false;
          break;
        }
        umma_fence_after();
        const uint32_t ta = taddr0 + buf * kAccCols;
        // eight pieces of 16 columns, the next one on its way while one is added
        uint32_t u[2][16];
        umma_ld16(ta + c0, u[0]);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          umma_ld_wait(u[p & 1]);
          if (p < 7) umma_ld16(ta + (p + 1 < 4 ? c0 : c1) + 16 * ((p + 1) & 3), u[(p + 1) & 1]);
          if (p == 7) {
            umma_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(buf));
          }
          promote16(u[p & 1], p < 4 ? s0 : s1, (p < 4 ? acc0 : acc1) + 8 * (p & 3));
        }
        if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
      }
      if (!ok) break;
      if constexpr (SPLIT > 1) {
        // Each rank finishes the rows of 4 / SPLIT lane quadrants: every warp of another
        // quadrant sends its sums there, into the stages, once the receiver's MMAs have read
        // them for the last time (a cluster has one tile) and its commit says so here.
        constexpr int kOwn = 4 / SPLIT;
        const int owner = quad / kOwn;
        if (threadIdx.x == 64) mbar_arrive_expect_tx(red_bar, (SPLIT - 1) * kOwn * 2 * kWarpSums);
        awaited = true;
        __syncwarp();
        // The slot of sender `from` for this warp: its distance behind the owner, the warp's
        // quadrant in the owner's, its half of the columns.
        auto slot = [&](int dist) {
          return stage_base + (((dist - 1) * kOwn + quad % kOwn) * 2 + half) * kWarpSums + lane * 16;
        };
        if (owner != rank) {
          ok = __all_sync(0xFFFFFFFFu, wait_bounded<true>(go_bar(owner), tile_ph, abort_flag, a.dev_status));
          if (ok) {
            const uint32_t dst = map_to_rank(smem_u32(slot((rank - owner + SPLIT) % SPLIT)), owner);
            const uint32_t bar = map_to_rank(red_bar, owner);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              st_async4(dst + j * 512, bar, acc0[2 * j].x, acc0[2 * j].y, acc0[2 * j + 1].x,
                        acc0[2 * j + 1].y);
              st_async4(dst + (16 + j) * 512, bar, acc1[2 * j].x, acc1[2 * j].y, acc1[2 * j + 1].x,
                        acc1[2 * j + 1].y);
            }
          }
        } else {
          ok = __all_sync(0xFFFFFFFFu, wait_bounded<true>(red_bar, tile_ph, abort_flag, a.dev_status));
          if (ok) {
#pragma unroll
            for (int i = 1; i < SPLIT; ++i) {
              const float4* in = reinterpret_cast<const float4*>(slot(i));
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float4 v = in[j * 32], w = in[(16 + j) * 32];
                acc0[2 * j].x += v.x; acc0[2 * j].y += v.y;
                acc0[2 * j + 1].x += v.z; acc0[2 * j + 1].y += v.w;
                acc1[2 * j].x += w.x; acc1[2 * j].y += w.y;
                acc1[2 * j + 1].x += w.z; acc1[2 * j + 1].y += w.w;
              }
            }
          }
        }
        tile_ph ^= 1u;
        if (!ok) break;
        if (owner != rank) continue;
      }
      if constexpr (SWIGLU) {
        // H of 64 columns in place of the gate sums, their largest magnitude, the
        // other half's through shared memory, then the group's codes
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          acc0[i].x = __fdividef(acc0[i].x, 1.0f + __expf(-acc0[i].x)) * acc1[i].x;
          acc0[i].y = __fdividef(acc0[i].y, 1.0f + __expf(-acc0[i].y)) * acc1[i].y;
          top = max(top, max(__float_as_uint(acc0[i].x) & 0x7FFFFFFFu,
                             __float_as_uint(acc0[i].y) & 0x7FFFFFFFu));
        }
        uint32_t* am = s_amax + parity * 256;
        am[half * 128 + r] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(amax_bar(quad));
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(amax_bar(quad), static_cast<uint32_t>(parity),
                                                  abort_flag, a.dev_status)))
          break;
        parity ^= 1;
        top = max(top, am[(half ^ 1) * 128 + r]);
        if (live) {
          const float s = scale_of(top);
          // One reciprocal a row instead of 64 divisions (H itself is known to fp32
          // rounding only; with the divisions the epilogue took 3 us a tile, a
          // fifth of the pass at K = 4096).  A scale near the type's smallest
          // values is taken 2^64 larger, so that its reciprocal stays finite.
          const float k = s < 0x1p-60f ? 0x1p64f : 1.0f;
          const float inv = __frcp_rn(s * k);
          if (top >= kAbsInf && half == 0) report(a.dev_status, MOE_DEV_NONFINITE_INPUT);
          if (half == 0) a.hs[row * a.GN + tl.nb] = s;
          const int n0 = tl.nb * 128 + 64 * half;
          uint8_t* dst = a.hq + row * a.N + n0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // 32 codes; N is a multiple of 16
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 x = acc0[16 * j + 2 * i], z = acc0[16 * j + 2 * i + 1];
              const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                  make_float2(x.x * k * inv, x.y * k * inv), __NV_SATFINITE, __NV_E4M3);
              const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                  make_float2(z.x * k * inv, z.y * k * inv), __NV_SATFINITE, __NV_E4M3);
              p[i] = lo | (hi << 16);
            }
            if (n0 + 32 * j + 16 < a.N)
              store32(dst + 32 * j, p);
            else if (n0 + 32 * j < a.N)
              *reinterpret_cast<uint4*>(dst + 32 * j) = make_uint4(p[0], p[1], p[2], p[3]);
          }
        }
      } else if (live) {
        const int n0 = tl.nb * 256 + 128 * half;
        uint16_t* dst = a.y + row * a.N + n0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // 16 columns; N is a multiple of 16
          if (n0 + 16 * j < a.N) {
            const float2* v = j < 4 ? acc0 + 8 * j : acc1 + 8 * (j - 4);
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = pack_bf16x2(v[i].x, v[i].y);
            store32(dst + 16 * j, p);
          }
        }
      }
    }
  }

  // ---- teardown ----
  __syncwarp();
  umma_fence_before();
  if constexpr (SPLIT > 1) {
    cluster_sync();  // no CTA leaves while a partner may still reach it
    // (after a wait that gave up: nor before the sums that were on their way)
    if (threadIdx.x == 64 && awaited && *abort_flag) wait_drain(red_bar, 0);
  } else {
    __syncthreads();
  }
  umma_fence_after();
  if (warp == 1) {
    __syncwarp();
    umma_dealloc(tmem, 2 * kAccCols);
  }
  pdl_trigger();
}

constexpr int kSmemBytes =
    1024 + kStages * kStageBytes + kBars * 8 + 512 * 4 + table_bytes(kMaxSeg);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(kStages * kStageBytes >= 6 * kWarpSums, "a partner's sums fit the stages");

// ------------------------------- few rows a segment --------------------------
// Decode-sized segments stream the weights; a 128-row tile would stage and sum
// mostly foreign rows.  Here the weights are the M operand: two [128 x 128] weight
// boxes a stage (gate and up of 128 columns, or 256 columns of down) against a box
// of NT rows (16 or 32), so D^T is [2 x 128 columns] x [NT rows].  A promotion thread owns one
// weight column and NT sums; the rows' scales come to it by shuffles.  Eight
// promotion warps: the four lane quadrants of either box.  Four tensor-memory
// buffers of 2 x NT columns.
//
// With SPLIT = 2 or 4 a cluster of that many CTAs shares a tile, each taking its part
// of the reduction blocks; the others hand their sums to rank 0 through distributed
// shared memory and rank 0 adds them in rank order.  One SM streams about 60 GB/s, so
// where the tiles are fewer than half (a fifth) of the SMs the number of SMs that
// stream sets the time: see launch_pass.
//
// CHAINED (down pass issued by moe_grouped_swiglu_w8 right behind its gate/up pass):
// the segment table and the first stages' weights, which the gate/up pass does not
// write, are read before waiting for it.

constexpr int kFewBufs = 4;

template <bool SWIGLU, int NT, int SPLIT>
struct Few {
  // Two CTAs an SM where two stages each fit: one's set-up, epilogue and launch
  // overlap the other's streaming (decode bucket 102 -> 98 us).  The passes split in
  // two share an SM with each other: a gate/up CTA of three stages beside a down CTA
  // that holds its first two.
  static constexpr int kPerSm = SPLIT == 4 || (NT == 32 && SPLIT == 2) ? 1 : 2;
  static constexpr int kBudget = (kPerSm == 2 ? 113 : 227) * 1024;
  static constexpr int kStageBytes = 2 * kBBox + NT * kBK;
  // the other ranks' sums ([SPLIT - 1][2][NT / 4][128][4]), and the up sums for the gate
  // warps (in rank 1's second half, or a buffer of their own)
  static constexpr int kRedBytes = (SPLIT - 1) * 2 * NT * 128 * 4;
  static constexpr int kUpBytes = SWIGLU && SPLIT == 1 ? NT * 128 * 4 : 0;
  static constexpr int kTopBytes = 2 * 4 * NT * 4;
  // bars: full[S], empty[S], tfull[4], tempty[4], upfull, upfree, top, red, redfree, drain
  static constexpr int kFixed = 1024 + kUpBytes + kRedBytes + kTopBytes + 64 * 8;  // + the table
  static constexpr int kStages = NT == 16 && SPLIT == 2 ? (SWIGLU ? 3 : 2)
                                     : (kBudget - kFixed - table_bytes(kMaxSeg)) / kStageBytes;
  static constexpr int kBars = 2 * kStages + 2 * kFewBufs + 6;
  static constexpr int kTmem = kFewBufs * 2 * NT;
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
  static_assert(kBars <= 64 && kStages >= 2, "stages");
  static_assert(kSmem + table_bytes(kMaxSeg) <= 227 * 1024, "shared memory");
  static_assert(kTmem * kPerSm <= 512 && kTmem >= 32, "tensor memory");
};

template <bool SWIGLU, int NT, int SPLIT>
__global__ void __launch_bounds__(kThreads, Few<SWIGLU, NT, SPLIT>::kPerSm)
grouped_w8_few_kernel(const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_w0,
                      const __grid_constant__ CUtensorMap map_w1, const W8Args a) {
  using F = Few<SWIGLU, NT, SPLIT>;
  constexpr int kStages = F::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stage_base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage_base + kStages * F::kStageBytes);
  float4* s_red = reinterpret_cast<float4*>(bars + 64);                       // [SPLIT-1][2][NT/4][128]
  float4* s_up = SPLIT > 1 ? s_red + NT / 4 * 128 : s_red;                    // [NT/4][128]
  uint32_t* s_top = reinterpret_cast<uint32_t*>(s_red + (F::kRedBytes + F::kUpBytes) / 16);  // [2][4][NT]
  const Table tb = carve_table(reinterpret_cast<int*>(s_top + F::kTopBytes / 4), a.n_seg);
  volatile int* abort_flag = tb.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kCols = SWIGLU ? 128 : 256;  // output columns per tile
  const int n_blocks = (a.N + kCols - 1) / kCols;
  const int rank = SPLIT > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int group = static_cast<int>(blockIdx.x) / SPLIT, groups = static_cast<int>(gridDim.x) / SPLIT;
  const int kb0 = rank * a.GK / SPLIT, kb1 = (rank + 1) * a.GK / SPLIT;

  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + kStages + s); };
  auto tfull_bar = [&](int b) { return smem_u32(bars + 2 * kStages + b); };
  auto tempty_bar = [&](int b) { return smem_u32(bars + 2 * kStages + kFewBufs + b); };
  auto bar_of = [&](int i) { return smem_u32(bars + 2 * kStages + 2 * kFewBufs + i); };
  const uint32_t up_full = bar_of(0), up_free = bar_of(1), top_bar = bar_of(2), red_full = bar_of(3),
                 red_free = bar_of(4), drain_bar = bar_of(5);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < kFewBufs; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 8);
    }
    mbar_init(up_full, 4);
    mbar_init(up_free, 4);
    mbar_init(top_bar, 4);
    mbar_init(red_full, 1);
    mbar_init(red_free, SWIGLU ? 128 : 256);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w0)) : "memory");
    if (SWIGLU)
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w1)) : "memory");
  }
  if (warp == 1) umma_alloc(smem_u32(tb.tmem_slot), F::kTmem);
  if (!a.chained) pdl_wait();
  // the grid fits the GPU at once: all of it is resident once all have passed here
  if (SWIGLU && SPLIT == 1) pdl_trigger();
  if (threadIdx.x >= 64 && threadIdx.x < 192) build_table(a, NT, n_blocks, threadIdx.x - 64, tb);
  umma_fence_before();
  if constexpr (SPLIT > 1) cluster_sync();  // the partner's barriers are initialised
  else __syncthreads();
  umma_fence_after();
  bool awaited = false;  // the partners' sums, in phase
  uint32_t awaited_ph = 0;
  const uint32_t tmem = *tb.tmem_slot;
  const int total = tb.start[a.n_seg];

  if (warp == 0) {
    if (lane == 0) {
      // ---- TMA producer ----
      auto load_weights = [&](const Tile& tl, int kb, int s) {
        const uint32_t st = smem_u32(stage_base + s * F::kStageBytes);
        mbar_arrive_expect_tx(full_bar(s), F::kStageBytes);
        tma_load_3d(st, &map_w0, full_bar(s), kb * kBK, tl.nb * kCols, tl.seg);
        tma_load_3d(st + kBBox, SWIGLU ? &map_w1 : &map_w0, full_bar(s), kb * kBK,
                    SWIGLU ? tl.nb * kCols : tl.nb * kCols + 128, tl.seg);
      };
      int s = 0, ahead = 0;
      uint32_t ph = 0;
      bool ok = true;
      if (a.chained) {
        if (group < total) {
          const Tile tl = tile_of(group, tb, a.n_seg, NT, n_blocks, a.m_outer);
          ahead = min(kStages, kb1 - kb0);
          for (int i = 0; i < ahead; ++i) load_weights(tl, kb0 + i, i);
        }
        pdl_wait();  // the rows are the previous pass's output
      }
      for (int t = group; t < total && ok; t += groups) {
        const Tile tl = tile_of(t, tb, a.n_seg, NT, n_blocks, a.m_outer);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (ahead > 0) {
            --ahead;
          } else {
            if (!wait_bounded(empty_bar(s), ph ^ 1u, abort_flag, a.dev_status)) { ok = false; break; }
            load_weights(tl, kb, s);
          }
          tma_load_2d(smem_u32(stage_base + s * F::kStageBytes + 2 * kBBox), &map_x, full_bar(s),
                      kb * kBK, tl.row0);
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
      // Split passes, one tile a CTA: all of its loads are under way, so a down pass
      // behind it may come and load its first weights while the sums, SiLU and codes are
      // finished (let in at the start, its loads delayed these: one token 18.2 -> 16.3 us).
      if (SWIGLU && SPLIT > 1) pdl_trigger();
      if (!ok) {
        for (int i = 0; i < kStages; ++i) {
          if (--s < 0) { s = kStages - 1; ph ^= 1u; }
          wait_drain(full_bar(s), ph);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- MMA issuer: gate (or the first 128 columns), then up (the second) ----
      constexpr uint32_t idesc = umma_idesc_e4m3(128, NT);
      int s = 0, buf = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true, issued = false;
      for (int t = group; t < total && ok; t += groups) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bounded(tempty_bar(buf), acc_ph ^ 1u, abort_flag, a.dev_status) ||
              !wait_bounded(full_bar(s), ph, abort_flag, a.dev_status)) {
            ok = false;
            break;
          }
          umma_fence_after();
          const uint32_t st = smem_u32(stage_base + s * F::kStageBytes);
          const uint32_t dst = tmem + buf * (2 * NT);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f8(dst + h * NT, umma_desc(st + h * kBBox + kk * 32),
                      umma_desc(st + 2 * kBBox + kk * 32), idesc, kk > 0);
          issued = true;
          umma_commit(empty_bar(s));
          umma_commit(tfull_bar(buf));
          if (++s == kStages) { s = 0; ph ^= 1u; }
          if (++buf == kFewBufs) { buf = 0; acc_ph ^= 1u; }
        }
      }
      if (!ok && issued) {
        umma_commit(drain_bar);
        wait_drain(drain_bar, 0);
      }
    }
  } else {
    // ---- promotion and epilogue ----
    if (a.chained) pdl_wait();  // the rows' scales
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int m = quad * 32 + lane;
    const uint32_t taddr0 = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * NT;
    constexpr int kPer = (NT + 31) / 32;  // rows whose scales this lane holds
    auto free_partners = [&]() {
#pragma unroll
      for (int o = 1; o < SPLIT; ++o) mbar_arrive_cluster(map_to_rank(red_free, o));
    };
    int buf = 0;
    uint32_t acc_ph = 0, tile_ph = 0;
    bool ok = true;
    for (int t = group; t < total; t += groups, tile_ph ^= 1u) {
      const Tile tl = tile_of(t, tb, a.n_seg, NT, n_blocks, a.m_outer);
      if (SPLIT > 1 && rank == 0 && threadIdx.x == 64)
        mbar_arrive_expect_tx(red_full, (SPLIT - 1) * 2 * 128 * 16 * ((min(tl.rows, NT) + 3) / 4));
      awaited = true;
      awaited_ph = tile_ph;
      const int nblk = SWIGLU ? tl.nb : min(2 * tl.nb + half, a.GN - 1);
      const float* ws = (SWIGLU && half ? a.bs1 : a.bs0) +
                        (static_cast<int64_t>(tl.seg) * a.GN + nblk) * a.GK;
      const float* xs[kPer];
      float x[kPer], w = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        xs[i] = a.as + static_cast<int64_t>(min(tl.row0 + min(lane + 32 * i, NT - 1), a.max_rows - 1)) * a.GK;
        x[i] = kb0 < kb1 ? __ldg(xs[i] + kb0) : 0.0f;
      }
      if (kb0 < kb1) w = __ldg(ws + kb0);
      float acc[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = 0.0f;
      for (int kb = kb0; kb < kb1; ++kb) {
        float p[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) p[i] = x[i] * w;
        if (kb + 1 < kb1) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) x[i] = __ldg(xs[i] + kb + 1);
          w = __ldg(ws + kb + 1);
        }
        if (!__all_sync(0xFFFFFFFFu,
                        wait_bounded(tfull_bar(buf), acc_ph, abort_flag, a.dev_status))) {
          ok = false;
          break;
        }
        umma_fence_after();
        const uint32_t ta = taddr0 + buf * (2 * NT);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          uint32_t u[16];
          umma_ld16(ta + c, u);
          umma_ld_wait(u);
          if (c + 16 == NT) {
            umma_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(buf));
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[c + j] = fmaf(__uint_as_float(u[j]),
                              __shfl_sync(0xFFFFFFFFu, p[(c + j) / 32], (c + j) & 31), acc[c + j]);
        }
        if (++buf == kFewBufs) { buf = 0; acc_ph ^= 1u; }
      }
      if (!ok) break;
      const bool more = t + groups < total;  // the other ranks will need the buffer again
      if constexpr (SPLIT > 1) {
        float4* mine = s_red + half * (NT / 4 * 128) + m;
        if (rank > 0) {
          if (!__all_sync(0xFFFFFFFFu, wait_bounded<true>(red_free, tile_ph ^ 1u, abort_flag, a.dev_status)))
            break;
          const uint32_t dst = map_to_rank(smem_u32(mine + (rank - 1) * (NT / 2 * 128)), 0);
          const uint32_t bar = map_to_rank(red_full, 0);
#pragma unroll
          for (int j = 0; j < NT; j += 4)
            if (j < tl.rows) st_async4(dst + j * 512, bar, acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
          continue;
        }
        if (!__all_sync(0xFFFFFFFFu, wait_bounded<true>(red_full, tile_ph, abort_flag, a.dev_status)))
          break;
#pragma unroll
        for (int o = 0; o < SPLIT - 1; ++o)
#pragma unroll
          for (int j = 0; j < NT; j += 4)
            if (j < tl.rows) {
              const float4 v = mine[(o * (NT / 2) + j / 4) * 128];
              acc[j] += v.x; acc[j + 1] += v.y; acc[j + 2] += v.z; acc[j + 3] += v.w;
            }
        if (!SWIGLU && more) free_partners();
      }
      if constexpr (SWIGLU) {
        if (half == 1) {
          if (!__all_sync(0xFFFFFFFFu, wait_bounded(up_free, tile_ph ^ 1u, abort_flag, a.dev_status)))
            break;
#pragma unroll
          for (int j = 0; j < NT; j += 4)
            if (j < tl.rows)
              s_up[j / 4 * 128 + m] = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
          __syncwarp();
          if (lane == 0) mbar_arrive(up_full);
          continue;
        }
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(up_full, tile_ph, abort_flag, a.dev_status))) break;
        uint32_t* tops = s_top + tile_ph * (4 * NT);
#pragma unroll
        for (int j = 0; j < NT; j += 4) {
          if (j >= tl.rows) break;
          const float4 v = s_up[j / 4 * 128 + m];
          const float up[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[j + i] = __fdividef(acc[j + i], 1.0f + __expf(-acc[j + i])) * up[i];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j >= tl.rows) break;
          const uint32_t v = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(acc[j]) & 0x7FFFFFFFu);
          if (lane == (j & 31)) tops[quad * NT + j] = v;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(up_free);
          mbar_arrive(top_bar);
        }
        if (SPLIT > 1 && more) free_partners();
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(top_bar, tile_ph, abort_flag, a.dev_status))) break;
        float k[kPer], inv[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int j = min(lane + 32 * i, NT - 1);
          const uint32_t top = max(max(tops[j], tops[NT + j]), max(tops[2 * NT + j], tops[3 * NT + j]));
          const float s = scale_of(top);
          k[i] = s < 0x1p-60f ? 0x1p64f : 1.0f;  // as in the 128-row kernel
          inv[i] = __frcp_rn(s * k[i]);
          if (quad == 0 && lane + 32 * i < tl.rows) {
            if (top >= kAbsInf) report(a.dev_status, MOE_DEV_NONFINITE_INPUT);
            a.hs[static_cast<int64_t>(tl.row0 + j) * a.GN + tl.nb] = s;
          }
        }
        const int n = tl.nb * 128 + m;
        uint8_t* dst = a.hq + static_cast<int64_t>(tl.row0) * a.N + n;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (j >= tl.rows) break;
          const float kj = __shfl_sync(0xFFFFFFFFu, k[j / 32], j & 31);
          const float ij = __shfl_sync(0xFFFFFFFFu, inv[j / 32], j & 31);
          if (n < a.N)
            dst[static_cast<int64_t>(j) * a.N] =
                __nv_cvt_float_to_fp8(acc[j] * kj * ij, __NV_SATFINITE, __NV_E4M3);
        }
      } else {
        const int n = tl.nb * 256 + half * 128 + m;
        uint16_t* dst = a.y + static_cast<int64_t>(tl.row0) * a.N + n;
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (j < tl.rows && n < a.N)
            dst[static_cast<int64_t>(j) * a.N] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[j]));
      }
    }
  }

  // ---- teardown ----
  __syncwarp();
  umma_fence_before();
  if constexpr (SPLIT > 1) {
    cluster_sync();  // no CTA leaves while its partner may still reach it
    // (after a wait that gave up: nor before the sums that were on their way)
    if (threadIdx.x == 64 && rank == 0 && awaited && *abort_flag) wait_drain(red_full, awaited_ph);
  } else {
    __syncthreads();
  }
  umma_fence_after();
  if (warp == 1) {
    __syncwarp();
    umma_dealloc(tmem, F::kTmem);
  }
  pdl_trigger();
}

// ------------------------------ weight quantization --------------------------

// One block per 128 x 128 weight block: w [K, N] bf16 -> codes [N, K] and a scale.
// 128 experts of 2048 x 768: 375 us, 1.6 TB/s, what bounds it not looked into: it runs once
// per set of weights.
__global__ void __launch_bounds__(256)
quantize_weights_kernel(int K, int N, const uint16_t* __restrict__ w, uint8_t* __restrict__ q,
                        float* __restrict__ scales, uint32_t* __restrict__ dev_status) {
  __shared__ uint32_t s_top[8];
  __shared__ __align__(16) uint8_t s_q[128][144];  // codes [n][k], rows padded by 16
  pdl_wait();
  const int n0 = blockIdx.x * 128, k0 = blockIdx.y * 128;
  const int64_t seg = blockIdx.z;
  const int tid = threadIdx.x, col = (tid & 15) * 8, kr = tid >> 4;
  const uint16_t* src = w + seg * K * N;
  uint4 v[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = k0 + kr + 16 * i;
    v[i] = k < K && n0 + col < N
               ? __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(k) * N + n0 + col))
               : make_uint4(0, 0, 0, 0);
    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      top = max(top, (x[j] << 16) & 0x7FFFFFFFu);
      top = max(top, x[j] & 0x7FFF0000u);
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, s_top[i]);
  const float s = scale_of(top);
  if (tid == 0) {
    if (top >= kAbsInf) report(dev_status, MOE_DEV_NONFINITE_INPUT);
    scales[(seg * gridDim.x + blockIdx.x) * gridDim.y + blockIdx.y] = s;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      s_q[col + j][kr + 16 * i] =
          __nv_cvt_float_to_fp8(__fdiv_rn(f[j], s), __NV_SATFINITE, __NV_E4M3);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = (tid >> 3) + 32 * i, k = (tid & 7) * 16;
    if (n0 + n < N && k0 + k < K)
      *reinterpret_cast<uint4*>(q + (seg * N + n0 + n) * K + k0 + k) =
          *reinterpret_cast<const uint4*>(&s_q[n][k]);
  }
  pdl_trigger();
}

// ------------------------------ host side ------------------------------------

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Codes [rows, K] with boxes of box_rows x 128, zero-filled past either edge.
bool map_rows(CUtensorMap* m, const void* base, uint64_t rows, uint64_t K, uint32_t box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {K, rows};
  const cuuint64_t strides[1] = {K};
  const cuuint32_t box[2] = {kBK, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Weight codes [n_seg, N, K]: a dimension of its own for the segment, so a box that
// passes N is filled with zeros and not with the next segment's rows.
bool map_weights(CUtensorMap* m, const void* base, uint64_t n_seg, uint64_t N, uint64_t K,
                 uint32_t box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {K, N, n_seg};
  const cuuint64_t strides[2] = {K, K * N};
  const cuuint32_t box[3] = {kBK, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// As in the bf16 pass: rows inner (one weight tile shared by neighbouring CTAs)
// unless a segment's rows outgrow the L2 while its weights fit.
int choose_m_outer(int32_t n_seg, int32_t max_rows, int32_t K, int64_t b_cols) {
  constexpr int64_t kL2Budget = 48ll << 20;
  const int64_t a_seg = static_cast<int64_t>(max_rows) / n_seg * K;
  const int64_t b_seg = static_cast<int64_t>(K) * b_cols;
  return a_seg > kL2Budget && b_seg <= kL2Budget ? 1 : 0;
}

moe_status check_shape(int32_t n_seg, int32_t K, int32_t N, int32_t max_rows) {
  if (n_seg <= 0 || K <= 0 || N <= 0 || max_rows < 0) return MOE_ERR_INVALID_ARG;
  if (n_seg > kMaxSeg || K % 16 != 0 || N % 16 != 0 || K > 65536 || N > 65536)
    return MOE_ERR_UNSUPPORTED;
  // row and tile numbers are 32-bit, a tile's last row among them
  if (max_rows > INT32_MAX - 1024 ||
      (static_cast<int64_t>(max_rows) / 16 + n_seg) * ceil_div(N, 128) >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Clusters that can be resident at once, read once per kernel and device.
template <typename Kernel>
int resident_clusters(Kernel kern, int cluster, int smem, std::mutex& mu, int (&cache)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sm_count() / cluster * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = sm_count() / cluster;
    }
    // one CTA an SM streams as fast as two
    cache[dev] = n < sm_count() / cluster ? n : sm_count() / cluster;
  }
  return cache[dev];
}

// The library's launch (programmatic dependent launch), with clusters of `cluster` CTAs.
template <typename Kernel>
void launch_clustered(Kernel kern, unsigned grid, int smem, int cluster, cudaStream_t s,
                      const CUtensorMap& m, const CUtensorMap& m0, const CUtensorMap& m1,
                      const W8Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
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
  cudaLaunchKernelEx(&cfg, kern, m, m0, m1, a);
}

template <bool SWIGLU, int NT, int SPLIT>
moe_status launch_few(const CUtensorMap& mx, const CUtensorMap& m0, const CUtensorMap& m1,
                      const W8Args& a, cudaStream_t s) {
  using F = Few<SWIGLU, NT, SPLIT>;
  auto kern = grouped_w8_few_kernel<SWIGLU, NT, SPLIT>;
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, F::kSmem + table_bytes(kMaxSeg), mu, done)) return MOE_ERR_CUDA;
  unsigned grid = static_cast<unsigned>(F::kPerSm * sm_count());
  if constexpr (SPLIT > 1) {
    static std::mutex mu2;
    static int clusters[64] = {};
    const int n = resident_clusters(kern, SPLIT, F::kSmem + table_bytes(kMaxSeg), mu2, clusters);
    if (n <= 0) return MOE_ERR_CUDA;
    grid = static_cast<unsigned>(SPLIT * n);
  }
  launch_clustered(kern, grid, F::kSmem + table_bytes(a.n_seg), SPLIT, s, mx, m0, m1, a);
  return launch_status();
}

// The 128-row kernel; with SPLIT > 1 only where every cluster has one tile at most, else
// false and nothing launched.
template <bool SWIGLU, int SPLIT>
bool launch_rows(const CUtensorMap& ma, const CUtensorMap& m0, const CUtensorMap& m1,
                 const W8Args& a, int64_t most_tiles, cudaStream_t s, moe_status& st) {
  auto kern = grouped_w8_kernel<SWIGLU, SPLIT>;
  unsigned grid = static_cast<unsigned>(sm_count());
  static std::mutex mu;
  static bool done[64] = {};
  if (!opt_in(kern, kSmemBytes, mu, done)) {
    st = MOE_ERR_CUDA;
    return true;
  }
  if constexpr (SPLIT > 1) {
    static std::mutex mu2;
    static int clusters[64] = {};
    if (most_tiles > resident_clusters(kern, SPLIT, kSmemBytes, mu2, clusters)) return false;
    grid = static_cast<unsigned>(SPLIT * most_tiles);
  }
  launch_clustered(kern, grid, kSmemBytes, SPLIT, s, ma, m0, m1, a);
  st = launch_status();
  return true;
}

// Rows per tile by the average rows of a segment: 16 up to 8, 32 up to 16 (segments are
// uneven; a longer one takes several tiles), above that the 128-row kernel.  A single
// segment is as long as the batch: 16 up to 32 rows, else 128.  Measured (us of both
// passes, 16 / 32 / 128 rows; 64 was slower than 128 everywhere): 128 experts,
// 2048 x 768: average 8: 93 / 98 / 102, 16: 106 / 100 / 105, 32: 142 / 114 / 117; 32 experts,
// 4096 x 2048: 8: 117 / 123 / 139, 16: 144 / 130 / 142, 24: 170 / 161 / 144; eight experts,
// 4096 x 1024: 8: 24 / 26 / 27, 16: 35 / 28 / 26, 32: 51 / 38 / 28; one expert, 7168 x 2048:
// 32 rows 25 / 33 / 27, 48: 37 / 33 / 27, 128: 57 / 40 / 27.
int choose_rows(int32_t n_seg, int32_t max_rows) {
  if (n_seg == 1) return max_rows <= 32 ? 16 : kBM;
  const int32_t avg = max_rows / n_seg;
  return avg <= 8 ? 16 : avg <= 16 ? 32 : kBM;
}

template <bool SWIGLU>
moe_status launch_pass(W8Args a, const void* x, const void* b0, const void* b1, bool chained,
                       cudaStream_t s) {
  const int nt = choose_rows(a.n_seg, a.max_rows);
  CUtensorMap ma, m0, m1;
  if (!map_rows(&ma, x, a.max_rows, a.K, nt) || !map_weights(&m0, b0, a.n_seg, a.N, a.K, 128) ||
      !map_weights(&m1, b1, a.n_seg, a.N, a.K, 128))
    return MOE_ERR_CUDA;
  if (nt < kBM) {
    a.chained = chained;
    a.m_outer = 0;
    // Tiles that hold rows, at most.  The reduction split over 1 / 2 / 4 CTAs, us of one pass
    // (one segment, 16-row tiles).  Gate/up, K = 2048: 16 tiles 14.6 / 9.8 / 8.0, 32: 15.5 /
    // 10.6 / 9.5, 40: 15.6 / 10.9 / 12.6, 64: 16.5 / 11.9 / 13.0; K = 7168: 16: 43.0 / 20.4 /
    // 13.9, 32: 43.4 / 21.1 / 15.2, 40: 43.9 / 21.5 / 25.3, 64: 45.6 / 24.5 / 25.8.  Down, 28
    // tiles, K = 2048: 14.8 / 11.0 / 9.0.  (So four would serve up to the 36 clusters that one
    // round holds; the rule stops at a fifth of the SMs, 30 tiles.)  From half of the SMs on
    // the split only adds the hand-over: both passes at 96 tiles 22 / 24 / 29.  Short reductions
    // gain little or lose: down, 64 tiles of eight segments, K = 256: 4.9 / 6.3, 768: 9.3 / 9.3,
    // 1024: 10.7 / 10.1.
    const int64_t tiles = std::min<int64_t>(a.n_seg, a.max_rows) * ceil_div(a.N, SWIGLU ? 128 : 256);
    const int split = 5 * tiles <= sm_count() && a.GK >= 8 ? 4 : 2 * tiles <= sm_count() && a.GK >= 2 ? 2 : 1;
    if (nt == 16) {
      if (split == 4) return launch_few<SWIGLU, 16, 4>(ma, m0, m1, a, s);
      if (split == 2) return launch_few<SWIGLU, 16, 2>(ma, m0, m1, a, s);
      return launch_few<SWIGLU, 16, 1>(ma, m0, m1, a, s);
    }
    // (32-row tiles have no split over four.  Gate/up, eight segments of 12 rows, 1 / 2 / 4
    // CTAs: 16 tiles, K = 2048 15.4 / 10.9 / 9.0, K = 7168 43.2 / 22.6 / 15.4.)
    if (split > 1) return launch_few<SWIGLU, 32, 2>(ma, m0, m1, a, s);
    return launch_few<SWIGLU, 32, 1>(ma, m0, m1, a, s);
  }
  // 128-row tiles, at most (each segment may end one).  From 16 blocks on the reduction is
  // split over the largest cluster of which one round holds them all (us of both passes,
  // 1 / 2 / 4 CTAs): one expert, 7168 x 2048, 128 rows: 41 / 32 / 27; 4096 x 14336:
  // 83 / 62 / 51; 2048 x 2048: 23.4 / 21.8 / 20.9; with 8 blocks it only adds the hand-over
  // (eight experts, 1024 x 1024, 128 rows each: 17.5 / 18.7).
  const int64_t segs = std::min<int64_t>(a.n_seg, a.max_rows);
  const int64_t tiles = (a.max_rows + 127 * segs) / 128 * ceil_div(a.N, SWIGLU ? 128 : 256);
  moe_status st = MOE_OK;
  if (a.GK >= 16) {
    if (launch_rows<SWIGLU, 4>(ma, m0, m1, a, tiles, s, st)) return st;
    if (launch_rows<SWIGLU, 2>(ma, m0, m1, a, tiles, s, st)) return st;
  }
  launch_rows<SWIGLU, 1>(ma, m0, m1, a, tiles, s, st);
  return st;
}

struct Pass {
  int32_t n_seg, K, N, max_rows;
  const int32_t *seg_begin, *seg_count;
  const void* x;
  const float* xs;
  const void *w0, *w1;
  const float *s0, *s1;
};

moe_status check_pass(const Pass& p, bool swiglu) {
  const moe_status st = check_shape(p.n_seg, p.K, p.N, p.max_rows);
  if (st != MOE_OK || p.max_rows == 0) return st;
  if (p.seg_begin == nullptr || p.seg_count == nullptr || p.x == nullptr || p.xs == nullptr ||
      p.w0 == nullptr || p.s0 == nullptr || (swiglu && (p.w1 == nullptr || p.s1 == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(p.x) || !aligned16(p.w0) || !aligned16(p.w1) || !aligned4(p.xs) ||
      !aligned4(p.s0) || !aligned4(p.s1) || !aligned4(p.seg_begin) || !aligned4(p.seg_count))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

W8Args args_of(const Pass& p, uint32_t* dev_status, bool swiglu) {
  W8Args a = {};
  a.seg_begin = p.seg_begin;
  a.seg_count = p.seg_count;
  a.n_seg = p.n_seg;
  a.K = p.K;
  a.N = p.N;
  a.max_rows = p.max_rows;
  a.GK = static_cast<int>(ceil_div(p.K, 128));
  a.GN = static_cast<int>(ceil_div(p.N, 128));
  a.as = p.xs;
  a.bs0 = p.s0;
  a.bs1 = p.s1;
  a.dev_status = dev_status;
  a.m_outer = choose_m_outer(p.n_seg, p.max_rows, p.K, (swiglu ? 2ll : 1ll) * p.N);
  return a;
}

size_t hidden_offset(int64_t max_rows, int64_t I) {
  return static_cast<size_t>((max_rows * I + 255) & ~int64_t(255));
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_quantize_weights_fp8(int32_t n_seg, int32_t K, int32_t N, const moe_bf16* w,
                                            moe_fp8* q, float* scales, uint32_t* dev_status,
                                            moe_stream_t stream) {
  if (n_seg <= 0 || K <= 0 || N <= 0 || w == nullptr || q == nullptr || scales == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (n_seg > kMaxSeg || K % 16 != 0 || N % 16 != 0 || K > 65536 || N > 65536 || !aligned16(w) ||
      !aligned16(q) || !aligned4(scales))
    return MOE_ERR_UNSUPPORTED;
  launch(quantize_weights_kernel,
         dim3(static_cast<unsigned>(ceil_div(N, 128)), static_cast<unsigned>(ceil_div(K, 128)),
              static_cast<unsigned>(n_seg)),
         dim3(256), 0, as_cuda(stream), K, N, w, q, scales, dev_status);
  return launch_status();
}

MOE_API moe_status moe_grouped_gate_up_w8(int32_t n_seg, int32_t d, int32_t I, int32_t max_rows,
                                          const moe_fp8* xq, const float* xs,
                                          const int32_t* seg_begin, const int32_t* seg_count,
                                          const moe_fp8* wg_q, const float* wg_s,
                                          const moe_fp8* wu_q, const float* wu_s, moe_fp8* hq,
                                          float* hs, uint32_t* dev_status, moe_stream_t stream) {
  const Pass p = {n_seg, d, I, max_rows, seg_begin, seg_count, xq, xs, wg_q, wu_q, wg_s, wu_s};
  const moe_status st = check_pass(p, true);
  if (st != MOE_OK || max_rows == 0) return st;
  if (hq == nullptr || hs == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(hq) || !aligned4(hs)) return MOE_ERR_UNSUPPORTED;
  W8Args a = args_of(p, dev_status, true);
  a.hq = hq;
  a.hs = hs;
  return launch_pass<true>(a, xq, wg_q, wu_q, false, as_cuda(stream));
}

namespace {
moe_status down_pass(int32_t n_seg, int32_t I, int32_t d, int32_t max_rows, const moe_fp8* hq,
                     const float* hs, const int32_t* seg_begin, const int32_t* seg_count,
                     const moe_fp8* wd_q, const float* wd_s, moe_bf16* y, bool chained,
                     uint32_t* dev_status, moe_stream_t stream) {
  const Pass p = {n_seg, I, d, max_rows, seg_begin, seg_count, hq, hs, wd_q, nullptr, wd_s, nullptr};
  const moe_status st = check_pass(p, false);
  if (st != MOE_OK || max_rows == 0) return st;
  if (y == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y)) return MOE_ERR_UNSUPPORTED;
  W8Args a = args_of(p, dev_status, false);
  a.y = y;
  return launch_pass<false>(a, hq, wd_q, wd_q, chained, as_cuda(stream));
}
}  // namespace

MOE_API moe_status moe_grouped_down_w8(int32_t n_seg, int32_t I, int32_t d, int32_t max_rows,
                                       const moe_fp8* hq, const float* hs,
                                       const int32_t* seg_begin, const int32_t* seg_count,
                                       const moe_fp8* wd_q, const float* wd_s, moe_bf16* y,
                                       uint32_t* dev_status, moe_stream_t stream) {
  return down_pass(n_seg, I, d, max_rows, hq, hs, seg_begin, seg_count, wd_q, wd_s, y, false,
                   dev_status, stream);
}

MOE_API size_t moe_grouped_swiglu_w8_workspace_size(int32_t max_rows, int32_t I) {
  if (max_rows < 0 || I <= 0 || I % 16 != 0 || I > 65536) return 0;
  return hidden_offset(max_rows, I) +
         static_cast<size_t>(max_rows) * static_cast<size_t>(ceil_div(I, 128)) * sizeof(float) + 256;
}

MOE_API moe_status moe_grouped_swiglu_w8(int32_t n_seg, int32_t d, int32_t I, int32_t max_rows,
                                         const moe_fp8* xq, const float* xs,
                                         const int32_t* seg_begin, const int32_t* seg_count,
                                         const moe_fp8* wg_q, const float* wg_s,
                                         const moe_fp8* wu_q, const float* wu_s,
                                         const moe_fp8* wd_q, const float* wd_s, moe_bf16* y,
                                         void* ws, size_t ws_bytes, uint32_t* dev_status,
                                         moe_stream_t stream) {
  // everything is checked before the first launch
  const Pass up = {n_seg, d, I, max_rows, seg_begin, seg_count, xq, xs, wg_q, wu_q, wg_s, wu_s};
  moe_status st = check_pass(up, true);
  if (st == MOE_OK) st = check_shape(n_seg, I, d, max_rows);
  if (st != MOE_OK || max_rows == 0) return st;
  if (wd_q == nullptr || wd_s == nullptr || y == nullptr || ws == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(wd_q) || !aligned4(wd_s) || !aligned16(y) || !aligned16(ws))
    return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < moe_grouped_swiglu_w8_workspace_size(max_rows, I)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  moe_fp8* hq = static_cast<moe_fp8*>(ws);
  float* hs = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + hidden_offset(max_rows, I));
  st = moe_grouped_gate_up_w8(n_seg, d, I, max_rows, xq, xs, seg_begin, seg_count, wg_q, wg_s, wu_q,
                              wu_s, hq, hs, dev_status, stream);
  if (st != MOE_OK) return st;
  return down_pass(n_seg, I, d, max_rows, hq, hs, seg_begin, seg_count, wd_q, wd_s, y, true,
                   dev_status, stream);
}
