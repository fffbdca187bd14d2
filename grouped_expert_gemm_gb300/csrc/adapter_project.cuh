// The projection of the rows with their adapters' part: kernel and launch of one shape.
#pragma once

#include "adapter.cuh"

namespace moe {
namespace adapter {
namespace {

// --------------------------------- project -----------------------------------
//
// D^T = W^T X^T: the weight's columns are the M operand, the tokens N, so a decode batch is a
// narrow tile and the weight streams once.  Roles of the 320 threads:
//   warp 0       TMA producer: [64 k x 128] of the weight (16 KB) and [tokens x 64 k] of x, once or
//                (few tokens) twice a stage
//   warp 1       tensor memory; lane 0 issues the MMAs (K = 16)
//   warps 2..9   epilogue: warp (quad, sub) has the 16 weight columns at 32 quad + 16 sub
// The adapters' part is made by the epilogue warps, 32 tokens at a time: u B is r / d of the work
// and a run of one adapter may be one token long, where tcgen05's narrowest tile is 16 columns
// by 128 rows of the table.
//   32 tokens of one adapter, or of a few runs: mma.sync.  tcgen05's 16x256b loads give the accumulators in its
//     layout, 16 weight columns by 8 tokens, so the table (16 columns, in registers, transposed
//     by movmatrix, once a run) is multiplied with u onto the sums themselves, and every token
//     takes the result of its own run.  u is split into bf16 numbers by all warps together: two a
//     value (16 bits) for bf16 results, which keep eight, three (all 24) for fp32 ones.
//   256 tokens of one adapter of up to 32 ranks (pairs): the reduction goes on over the ranks, u as
//     value and remainder against the table twice, both laid down in shared memory by the
//     epilogue warps while the tile's MMAs run.  (Beside running MMAs the products above take
//     2,000 cycles for 32 tokens.)
//   otherwise: warp w takes tokens 4w .. 4w + 3, each with its own adapter's rows (four columns
//     a lane, fp32), through shared memory.
// Nothing of one request, not even 0 times an infinity, reaches another's rows.
//
// Shapes (launch_project has the rule):
//   pair   a cluster of two CTAs, 256 weight columns by 256 tokens (cta_group::2), two
//          accumulator buffers that fill the tensor memory
//   flat   one CTA, 128 weight columns by TN = 64 or 128 tokens; the adapters' part is made
//          while the MMAs run and waits in tensor memory.  S > 1: a cluster shares a tile, each
//          CTA a part of the reduction; the CTA of rank c finishes its S-th of the tokens and
//          gets the others' sums through distributed shared memory.
// fp32 results of long reductions are summed in pieces of kPiece: the tensor cores' own fp32
// sums lose 2^-26 a step (7168: 8e-6 of the result, in these pieces 4.6e-7).
// The weight, x and the tables are read before shrink has ended; u is waited for.

constexpr int kThreads = 320;
constexpr int kWBytes = 128 * 64 * 2;
constexpr int kWBox = 64 * 64 * 2;
constexpr int kPiece = 8;  // blocks of 64 to a piece of an fp32 result's reduction
constexpr int kMaxRank = 128;

// 32 tokens of u: [value, remainder(s)][32][r, padded to 16 and 8 more], so that eight rows of an
// ldmatrix lie in other banks.
__host__ __device__ constexpr int u_pitch(int rp) { return rp * 2 + 16; }
// 32 tokens of the adapters' part: [32][128 columns and 4 more] fp32.
constexpr int kPartPitch = 132;

constexpr int kMoreU = 128 * 128;
constexpr int kMoreTable = 2 * 32 * 128;

template <int TN, int S, int CG>
struct Shape {
  // Blocks of 64 k a stage.  Two where the weight streams for few tokens: half as many, larger
  // boxes of it (128 k x 64).
  static constexpr int kDepth = TN == 64 ? 2 : 1;
  static constexpr int kXBlock = TN / CG * 128;
  static constexpr int kXOff = kDepth * kWBytes;
  static constexpr int kStageBytes = kDepth * (kWBytes + kXBlock);
  static constexpr int kStages = CG == 2 ? 5 : TN == 128 ? (S == 1 ? 5 : 4) : 3;
  static constexpr int kOwn = TN / S;
  static constexpr int kRedBytes = (S - 1) * kOwn * 512;  // [S - 1][kOwn / 8][8][32] float4
  // (pair) the tile's further reduction: [128 tokens][64] of u, [2][32 ranks][64 columns] of the table
  static constexpr int kMoreBytes = CG == 2 ? kMoreU + kMoreTable : 0;
  // bf16 numbers a value of u (pairs have bf16 results alone), the bytes of 32 tokens of u or of the
  // adapters' part, and buffers of them: a cluster that shares a tile has one, and a CTA whose tokens
  // are 32 at most fills one buffer once.
  static constexpr int kParts = CG == 2 ? 2 : 3;
  static constexpr int kPieceBytes = (CG == 2 ? 18 : 26) * 1024;
  static constexpr int kPieces = S > 1 && kOwn <= 32 ? 1 : 2;
  // full[st], empty[st], tfull[2], tempty[2], group, red, drain, more
  static constexpr int kBars = 2 * kStages + 8;
  static constexpr int kTmem = CG == 2 ? 2 * TN : 4 * TN;  // two buffers, (flat) the sums
  static constexpr int kSmem =
      1024 + kStages * kStageBytes + kMoreBytes + kPieces * kPieceBytes + kRedBytes + kBars * 8 +
      3 * (kOwn + 20) * 4 + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kOwn % 8 == 0 && kTmem <= 512, "shape");
  static_assert(kPieceBytes >= kParts * 32 * u_pitch(kMaxRank) && kPieceBytes >= 32 * kPartPitch * 4, "pieces");
};

constexpr int kFew = -3;      // 32 tokens of up to kFewRuns runs
constexpr int kSeveral = -4;  // of more
constexpr int kFewRuns = 6;

// First token of tile t, and first weight column of this CTA's part of it.  (With tokens inner
// each block of columns starts at another block of tokens: one whose adapters cost more does not
// come to the same CTAs in every round.)
template <int TN, int CG>
__device__ __forceinline__ void tile_at(const ProjectArgs& a, int t, int rank, int& row0, int& n0) {
  const int nb = a.n_inner ? t % a.n_blocks : t / a.t_blocks;
  const int tb = a.n_inner ? t / a.n_blocks : (t % a.t_blocks + nb) % a.t_blocks;
  row0 = tb * TN;
  n0 = nb * 128 * CG + (CG == 2 ? rank * 128 : 0);
}

__device__ __forceinline__ void fma4(float4& acc, float u, const uint2& b) {
  acc.x = fmaf(u, __uint_as_float(b.x << 16), acc.x);
  acc.y = fmaf(u, __uint_as_float(b.x & 0xFFFF0000u), acc.y);
  acc.z = fmaf(u, __uint_as_float(b.y << 16), acc.z);
  acc.w = fmaf(u, __uint_as_float(b.y & 0xFFFF0000u), acc.w);
}

// acc += u B of four consecutive rows, columns n .. n + 3 of this lane; id: their adapters (rows
// without one stay).  32 loads of a lane are on their way at once: 32 ranks of one adapter, or
// eight of each of four (one row after the other, 16 ranks at a time, took three times as long).
__device__ __forceinline__ void expand(const ProjectArgs& a, const int (&id)[4], int row, int lane,
                                       int n, float4 (&acc)[4]) {
  const bool same = id[0] >= 0 && id[0] == id[1] && id[0] == id[2] && id[0] == id[3];
  const uint16_t* tab = a.table + n;
  const int64_t table_size = static_cast<int64_t>(a.r) * a.N;
  for (int c = 0; c < a.r; c += 32) {
    float u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = id[i] >= 0 && c + lane < a.r ? a.u[static_cast<int64_t>(row + i) * a.r + c + lane] : 0.0f;
    if (same) {
      uint2 v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j)
        v[j] = n < a.N && c + j < a.r ? __ldg(reinterpret_cast<const uint2*>(tab + id[0] * table_size +
                                                                             static_cast<int64_t>(c + j) * a.N))
                                      : make_uint2(0, 0);
#pragma unroll
      for (int j = 0; j < 32; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) fma4(acc[i], __shfl_sync(0xFFFFFFFFu, u[i], j), v[j]);
    } else {
      for (int k = 0; k < 32 && c + k < a.r; k += 8) {  // (r is a multiple of 8)
        uint2 v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[i][j] = n < a.N && id[i] >= 0
                          ? __ldg(reinterpret_cast<const uint2*>(tab + id[i] * table_size +
                                                                 static_cast<int64_t>(c + k + j) * a.N))
                          : make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) fma4(acc[i], __shfl_sync(0xFFFFFFFFu, u[i], k + j), v[i][j]);
      }
    }
  }
}

// What the rounding of four values to bf16 left of them.
__device__ __forceinline__ float4 left_of(const float4& f, uint32_t h0, uint32_t h1) {
  return make_float4(f.x - __uint_as_float(h0 << 16), f.y - __uint_as_float(h0 & 0xFFFF0000u),
                     f.z - __uint_as_float(h1 << 16), f.w - __uint_as_float(h1 & 0xFFFF0000u));
}

// Stores 16 weight columns from n by 8 G tokens from row (the layout of umma_ld_frag); id: the
// tokens'.
template <int G>
__device__ __forceinline__ void put_frags(const ProjectArgs& a, const float (&c)[G][4], int row, int n,
                                          const int* id, int lane) {
  const int g = lane >> 2, t4 = lane & 3;
  if (a.y_fp32) {
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (id[8 * i + 2 * t4 + e] != kOutside) {
          float* y = static_cast<float*>(a.y) + static_cast<int64_t>(row + 8 * i + 2 * t4 + e) * a.y_stride + n + g;
          if (n < a.N) y[0] = c[i][e];
          if (n + 8 < a.N) y[8] = c[i][2 + e];
        }
    return;
  }
  // rows become tokens: two 8 x 8 blocks transposed, then 4 columns to a lane
  uint32_t d[G][2], other[G];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    d[i][0] = pack_bf16x2(c[i][0], c[i][1]);
    d[i][1] = pack_bf16x2(c[i][2], c[i][3]);
  }
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(d[i][h]));
  const bool odd = t4 & 1;
#pragma unroll
  for (int i = 0; i < G; ++i) other[i] = __shfl_xor_sync(0xFFFFFFFFu, odd ? d[i][0] : d[i][1], 1);
  const int col = n + (odd ? 8 + 2 * (t4 - 1) : 2 * t4);
  uint16_t* y = static_cast<uint16_t*>(a.y) + static_cast<int64_t>(row + g) * a.y_stride + col;
#pragma unroll
  for (int i = 0; i < G; ++i)
    if (col < a.N && id[8 * i + g] != kOutside)
      *reinterpret_cast<uint2*>(y + 8 * i * a.y_stride) =
          odd ? make_uint2(other[i], d[i][1]) : make_uint2(d[i][0], other[i]);
}

// What the epilogue warps share.
struct Epilogue {
  uint8_t* piece;   // [kPieces][kPieceBytes]
  uint8_t* red;
  uint8_t* more;    // kMoreU, then kMoreTable bytes
  // Three of each, tile by tile: the next tile's are made while other warps may still be at the last.
  int* id;          // [3][kOwn]: adapter of a token
  int* whole;       // [3][8]: of 32 tokens the adapter of all, kNone where none has one, kFew or kSeveral
  uint32_t* starts; // [3][8]: where their runs start
  volatile int* abort_flag;
  uint32_t tfull, tempty, group_bar, red_bar, more_bar;  // (tfull and tempty: two barriers each)
  uint32_t tmem;
  int first, step, total, rank, k0, k1, piece_steps;
};

// The epilogue warps' work; RB: blocks of 16 ranks.
template <int TN, int S, int CG, int RB>
__device__ __forceinline__ void epilogue(const ProjectArgs& a, const Epilogue& s, int warp, int lane) {
  constexpr int kOwn = TN / S, kChunks = (kOwn + 31) / 32, kGroups = kOwn < 32 ? kOwn / 8 : 4;
  constexpr int kPieceBytes = Shape<TN, S, CG>::kPieceBytes;
  const bool whole_u = CG == 1 && a.y_fp32;  // u as three numbers
  constexpr int kQuads = 4 * RB;                              // groups of four values of a row of u
  constexpr int kLoads = (8 * kGroups * kQuads + 255) / 256;  // of them a thread
  constexpr int kPitch = u_pitch(16 * RB);
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int w = warp - 2, quad = warp & 3, sub = w >> 2, tid = threadIdx.x - 64;
  const int g = lane >> 2, t4 = lane & 3;
  const int m0 = 32 * quad + 16 * sub;
  const int own0 = S > 1 ? s.rank * kOwn : 0;
  const uint32_t taddr = s.tmem + (static_cast<uint32_t>(m0) << 16);
  const uint32_t sums = taddr + 2 * TN;  // (flat) [kOwn], or in pieces [TN]
  int buf = 0, par = 0, pb = 0;
  uint32_t acc_ph = 0, group_ph = 0;
  bool ok = true;
  // Barrier of the eight warps: false if one of them gave up.
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(s.group_bar);
    const bool all = __all_sync(kAll, wait_bounded(s.group_bar, group_ph, s.abort_flag, a.dev_status));
    group_ph ^= 1u;
    return all;
  };
  auto sums_ready = [&]() {
    const bool all = __all_sync(kAll, wait_bounded(s.tfull + 8 * buf, acc_ph, s.abort_flag, a.dev_status));
    umma_fence_after();
    return all;
  };
  auto sums_read = [&]() {
    umma_fence_before();
    __syncwarp();
    if (lane == 0) {
      if constexpr (CG == 2) mbar_arrive_cluster(map_to_rank(s.tempty + 8 * buf, 0));
      else mbar_arrive(s.tempty + 8 * buf);
    }
    if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
  };
  // 16 columns of the table of adapter `held`, mma.sync's first operand; with up to 64 ranks the
  // next run's are already on their way (`coming`, not yet transposed)
  constexpr bool kAhead = RB <= 4;
  uint32_t tab[RB][4], raw[kAhead ? RB : 1][4];
  int held = kNone, coming = kNone, table_n = -1;
  auto load_table = [&](uint32_t (&to)[RB][4], int e, int n) {
    const uint16_t* p = a.table + (static_cast<int64_t>(e) * a.r + g) * a.N + n + 2 * t4;
#pragma unroll
    for (int k = 0; k < RB; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // columns + 8 (q & 1), ranks + 8 (q >> 1)
        const int rank_q = 16 * k + 8 * (q >> 1);
        to[k][q] = n + 8 * (q & 1) < a.N && rank_q < a.r
                       ? __ldg(reinterpret_cast<const uint32_t*>(p + static_cast<int64_t>(rank_q) * a.N + 8 * (q & 1)))
                       : 0u;
      }
  };
  auto expect = [&](int e, int n) {  // adapter e is the next one
    if constexpr (kAhead) {
      if (e < 0 || e == held || e == coming) return;
      coming = e;
      load_table(raw, e, n);
    }
  };
  auto hold = [&](int e, int n) {
    if (e == held) return;
    if constexpr (kAhead) {
      if (e == coming) {
#pragma unroll
        for (int k = 0; k < RB; ++k)
#pragma unroll
          for (int q = 0; q < 4; ++q) tab[k][q] = raw[k][q];
        coming = kNone;
      } else {
        load_table(tab, e, n);
      }
    } else {
      load_table(tab, e, n);
    }
    held = e;
#pragma unroll
    for (int k = 0; k < RB; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(tab[k][q]));
  };
  // this thread's part of the u of 32 tokens, on its way
  float4 ahead[kLoads];
  auto fetch_u = [&](int row) {
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      const int i = tid + 256 * e, q = i % kQuads * 4;
      ahead[e] = i < 8 * kGroups * kQuads && q < a.r && row + i / kQuads < a.seg.T
                     ? *reinterpret_cast<const float4*>(a.u + static_cast<int64_t>(row + i / kQuads) * a.r + q)
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  };
  // this lane's row of the four 8 x 8 blocks of an ldmatrix of u (two of the values, two of what
  // their rounding left): mma.sync's second operand of 8 tokens and 16 ranks
  const uint32_t lu = smem_u32(s.piece) + (lane & 7) * kPitch + (lane & 8) * 2 + (lane & 16 ? 32 * kPitch : 0);

  // c += u B on the 32 tokens of a piece
  auto multiply = [&](float (&c)[kGroups][4], uint32_t at) {
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      uint32_t u[kGroups][4];
#pragma unroll
      for (int i = 0; i < kGroups; ++i) ldmatrix(u[i], at + 8 * i * kPitch + k * 32);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
          mma_16816(c[i], tab[k][0], tab[k][1], tab[k][2], tab[k][3], u[i][2 * h], u[i][2 * h + 1]);
      if (whole_u) {  // the third numbers of two groups of eight tokens at once
        const uint32_t third = at + 64 * kPitch - (lane & 16 ? 24 * kPitch : 0);
#pragma unroll
        for (int i = 0; i < kGroups; i += 2) {
          uint32_t l[4];
          ldmatrix(l, third + 8 * i * kPitch + k * 32);
          mma_16816(c[i], tab[k][0], tab[k][1], tab[k][2], tab[k][3], l[0], l[1]);
          mma_16816(c[i + 1], tab[k][0], tab[k][1], tab[k][2], tab[k][3], l[2], l[3]);
        }
      }
    }
  };

  // Whose are the tokens of tile t: warp w finds out for 32 of them.
  auto look = [&](int t, int to) {
    if (w < kChunks) {
      int row0, n0;
      tile_at<TN, CG>(a, t, s.rank, row0, n0);
      const int id = row_adapters(a.seg, row0 + own0 + 32 * w, lane);
      constexpr uint32_t kIn = kOwn < 32 ? (1u << (kOwn & 31)) - 1 : kAll;
      const uint32_t has = __ballot_sync(kAll, id >= 0) & kIn;
      const int before = __shfl_up_sync(kAll, id, 1);
      const uint32_t starts = __ballot_sync(kAll, id >= 0 && (lane == 0 || id != before)) & kIn;
      if (32 * w + lane < kOwn) s.id[to * kOwn + 32 * w + lane] = id;
      if (lane == 0) {
        s.starts[to * 8 + w] = starts;
        s.whole[to * 8 + w] =
            has == 0 ? kNone : has == kIn && starts == 1 ? id : __popc(starts) <= kFewRuns ? kFew : kSeveral;
      }
    }
    return meet();
  };
  // The adapter of a whole tile (kNone: not of one adapter, or too many ranks).
  constexpr bool kMore = CG == 2 && RB <= 2;
  auto tile_adapter = [&](int of) {
    if constexpr (!kMore) return kNone;
    const int e = s.whole[of * 8];
    bool same = e >= 0;
#pragma unroll
    for (int ch = 1; ch < kChunks; ++ch) same = same && s.whole[of * 8 + ch] == e;
    return same ? e : kNone;
  };
  // The further reduction of tile t, if it is of one adapter: this CTA's half of the tokens' u and
  // its columns of the table, both zero behind rank r, as the MMAs take them.  The issuer is told
  // either way.
  auto lay_more = [&](int t, int of) {
    if constexpr (kMore) {
      const int e = tile_adapter(of);
      if (e >= 0) {
        int row0, n0;
        tile_at<TN, CG>(a, t, s.rank, row0, n0);
        row0 += s.rank * 128;
#pragma unroll
        for (int i = tid; i < 128 * 4 * RB; i += 256) {  // four values of a token
          const int tok = i / (4 * RB), q = i % (4 * RB);
          const float4 f = 4 * q < a.r ? *reinterpret_cast<const float4*>(
                                             a.u + static_cast<int64_t>(row0 + tok) * a.r + 4 * q)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          const uint32_t h0 = pack_bf16x2(f.x, f.y), h1 = pack_bf16x2(f.z, f.w);
          const float4 d = left_of(f, h0, h1);
          const uint32_t l0 = pack_bf16x2(d.x, d.y), l1 = pack_bf16x2(d.z, d.w);
          // 16-byte chunks of a row of 128: the values' first, then (2 RB on) the remainders'
          uint8_t* row = s.more + tok * 128 + (q & 1) * 8;
          *reinterpret_cast<uint2*>(row + (((q >> 1) ^ (tok & 7)) << 4)) = make_uint2(h0, h1);
          *reinterpret_cast<uint2*>(row + (((2 * RB + (q >> 1)) ^ (tok & 7)) << 4)) = make_uint2(l0, l1);
        }
#pragma unroll
        for (int i = tid; i < 16 * RB * 16; i += 256) {  // eight columns of a rank
          const int k = i / 16, c = i % 16, col = n0 + 8 * c;
          const uint4 v = k < a.r && col < a.N
                              ? __ldg(reinterpret_cast<const uint4*>(
                                    a.table + (static_cast<int64_t>(e) * a.r + k) * a.N + col))
                              : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(s.more + kMoreU + (c >> 3) * (16 * RB * 128) + k * 128 +
                                    (((c & 7) ^ (k & 7)) << 4)) = v;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(s.more_bar, 0));
    }
  };

  if (s.first < s.total && !look(s.first, 0)) return;
  bool waited = false;
  for (int t = s.first; t < s.total; t += s.step) {
    int row0, n0;
    tile_at<TN, CG>(a, t, s.rank, row0, n0);
    const int n = n0 + m0, row_own = row0 + own0;
    int* ids = s.id + par * kOwn;
    int* whole = s.whole + par * 8;
    const int coming_up = par == 2 ? 0 : par + 1;
    const bool more = t + s.step < s.total;
    if (n != table_n) held = coming = kNone;  // other columns
    table_n = n;
    // the first adapter of 32 tokens that mma.sync takes
    auto first_of = [&](int ch) {
      return whole[ch] == kFew ? ids[32 * ch + __ffs(s.starts[par * 8 + ch]) - 1] : whole[ch];
    };
    const bool done = tile_adapter(par) >= 0;  // the adapter's part is in the sums already
    if (!done) expect(first_of(0), n);
    if (!waited) {
      pdl_wait();  // u; and what is written here may still be read by the kernels before
      waited = true;
      lay_more(t, par);
    }
    if (!done && (whole[0] >= 0 || whole[0] == kFew)) fetch_u(row_own);
    if (more && !look(t + s.step, coming_up)) break;
    if constexpr (CG == 2) {
      if (!sums_ready()) break;
      if (more) lay_more(t + s.step, coming_up);  // (this tile's MMAs have read theirs)
    }
#pragma unroll 1
    for (int ch = 0; ch < kChunks; ++ch) {
      __syncwarp();  // (behind the last tokens' masked stores: loads of sums want whole warps)
      const int j = 32 * ch, kind = done ? kNone : whole[ch];
      uint8_t* piece = s.piece + pb * kPieceBytes;
      const uint32_t at = lu + pb * kPieceBytes;
      if (kind >= 0 || kind == kFew) {
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const int i = tid + 256 * e;
          const float4 f = ahead[e];
          const uint32_t h0 = pack_bf16x2(f.x, f.y), h1 = pack_bf16x2(f.z, f.w);
          const float4 d = left_of(f, h0, h1);
          const uint32_t l0 = pack_bf16x2(d.x, d.y), l1 = pack_bf16x2(d.z, d.w);
          if (i < 8 * kGroups * kQuads) {
            uint8_t* dst = piece + i / kQuads * kPitch + i % kQuads * 8;
            *reinterpret_cast<uint2*>(dst) = make_uint2(h0, h1);
            *reinterpret_cast<uint2*>(dst + 32 * kPitch) = make_uint2(l0, l1);
            if (whole_u) {
              const float4 q = left_of(d, l0, l1);
              *reinterpret_cast<uint2*>(dst + 64 * kPitch) = make_uint2(pack_bf16x2(q.x, q.y), pack_bf16x2(q.z, q.w));
            }
          }
        }
        hold(first_of(ch), n);
      } else if (kind == kSeveral && 4 * w < kOwn - j) {
        int id[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = ids[j + 4 * w + i];
        float4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int row = row_own + j + 4 * w;
        expand(a, id, row, lane, n0 + 4 * lane, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(piece + ((4 * w + i) * kPartPitch + 4 * lane) * 4) = acc[i];
      }
      if (kind != kNone) {
        ok = meet();
        if (!ok) break;
        pb ^= 1;  // (the other piece's readers have all come here)
      }
      if (!done && ch + 1 < kChunks && (whole[ch + 1] >= 0 || whole[ch + 1] == kFew)) fetch_u(row_own + j + 32);
      float c[kGroups][4];
      if constexpr (CG == 2) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) umma_ld_frag(taddr + buf * TN + j + 8 * i, c[i]);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) umma_ld_frag_wait(c[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[i][e] = 0.0f;
      }
      if (kind >= 0) {
        multiply(c, at);
      } else if (kind == kFew) {
        uint32_t starts = s.starts[par * 8 + ch];
#pragma unroll 1
        while (starts != 0) {
          const int b = __ffs(starts) - 1, mine = ids[j + b];  // tokens from b on, as long as they are mine
          starts &= starts - 1;
          const int end = starts != 0 ? __ffs(starts) - 1 : 8 * kGroups;
          hold(mine, n);
          if (starts != 0) expect(ids[j + __ffs(starts) - 1], n);
          else if (ch + 1 < kChunks) expect(first_of(ch + 1), n);
          // all 32 tokens (four products side by side), and each keeps its own run's
          float d[kGroups][4];
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[i][e] = c[i][e];
          multiply(d, at);
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int tok = 8 * i + 2 * t4 + e;
              if (tok >= b && tok < end && ids[j + tok] == mine) {
                c[i][e] = d[i][e];
                c[i][2 + e] = d[i][2 + e];
              }
            }
        }
      } else if (kind == kSeveral) {
        const float* part = reinterpret_cast<const float*>(piece) + m0 + g;
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            c[i][e] += part[(8 * i + 2 * t4 + (e & 1)) * kPartPitch + 8 * (e >> 1)];
      }
      if constexpr (CG == 2) {
        put_frags<kGroups>(a, c, row_own + j, n, ids + j, lane);
      } else {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) umma_st_frag(sums + own0 + j + 8 * i, c[i]);
      }
    }
    if (!ok) break;
    if constexpr (CG == 2) {
      sums_read();
    } else {
      const bool pieces = s.k0 + s.piece_steps < s.k1;
      if (S > 1 && pieces) {  // the other tokens' sums start at zero
        const float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < TN; j += 8)
          if (j < own0 || j >= own0 + kOwn) umma_st_frag(sums + j, z);
      }
      umma_st_wait();
      // every piece but the last onto the sums
      for (int kp = s.k0; kp + s.piece_steps < s.k1; kp += s.piece_steps) {
        ok = sums_ready();
        if (!ok) break;
        for (int j = 0; j < TN; j += 32) {
          float c[4][4], q[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            umma_ld_frag(taddr + buf * TN + j + 8 * i, c[i]);
            umma_ld_frag(sums + j + 8 * i, q[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            umma_ld_frag_wait(c[i]);
            umma_ld_frag_wait(q[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[i][e] += q[i][e];
            umma_st_frag(sums + j + 8 * i, c[i]);
          }
        }
        umma_st_wait();
        sums_read();
      }
      if (!ok || !sums_ready()) break;
      if constexpr (S > 1) {
        for (int i = 1; i < S; ++i) {  // the partners' tokens first
          const int owner = (s.rank + i) % S;
          const uint32_t bar = map_to_rank(s.red_bar, owner);
          const uint32_t dst =
              map_to_rank(smem_u32(s.red + (S - 1 - i) * kOwn * 512 + w * 512 + lane * 16), owner);
          for (int j = 0; j < kOwn; j += 8) {
            float c[4];
            umma_ld_frag(taddr + buf * TN + owner * kOwn + j, c);
            umma_ld_frag_wait(c);
            if (pieces) {
              float q[4];
              umma_ld_frag(sums + owner * kOwn + j, q);
              umma_ld_frag_wait(q);
#pragma unroll
              for (int e = 0; e < 4; ++e) c[e] += q[e];
            }
            st_async4(dst + j * 512, bar, c[0], c[1], c[2], c[3]);
          }
        }
        if (!__all_sync(kAll, wait_bounded<true>(s.red_bar, 0, s.abort_flag, a.dev_status))) break;
      }
      for (int j = 0; j < kOwn; j += 8 * kGroups) {
        float c[kGroups][4], q[kGroups][4];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          umma_ld_frag(taddr + buf * TN + own0 + j + 8 * i, c[i]);
          umma_ld_frag(sums + own0 + j + 8 * i, q[i]);
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          umma_ld_frag_wait(c[i]);
          umma_ld_frag_wait(q[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) c[i][e] += q[i][e];
          if constexpr (S > 1) {
#pragma unroll
            for (int o = 0; o < S - 1; ++o) {
              const float4 p = *reinterpret_cast<const float4*>(s.red + o * kOwn * 512 + (j + 8 * i) * 512 +
                                                                w * 512 + lane * 16);
              c[i][0] += p.x; c[i][1] += p.y; c[i][2] += p.z; c[i][3] += p.w;
            }
          }
        }
        put_frags<kGroups>(a, c, row_own + j, n, ids + j, lane);
      }
      sums_read();
    }
    par = coming_up;
  }
}

template <int TN, int S, int CG, bool KMAJ>
__global__ void __launch_bounds__(kThreads, 1)
project_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
               const ProjectArgs a) {
  using F = Shape<TN, S, CG>;
  static_assert(CG == 1 || S == 1, "one kind of cluster");
  constexpr int kStages = F::kStages, kOwn = F::kOwn;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stage_base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_more = stage_base + kStages * F::kStageBytes;
  uint8_t* s_piece = s_more + F::kMoreBytes;
  uint8_t* s_red = s_piece + F::kPieces * F::kPieceBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_red + F::kRedBytes);
  int* s_id = reinterpret_cast<int*>(bars + F::kBars);
  int* s_whole = s_id + 3 * kOwn;
  uint32_t* s_starts = reinterpret_cast<uint32_t*>(s_whole + 3 * 8);
  volatile int* abort_flag = s_whole + 6 * 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_whole + 6 * 8) + 1;
  uint32_t* ring_end = tmem_slot + 1;  // where the producer stopped, and whether MMAs were issued
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kCluster = S * CG;
  const int rank = kCluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const bool leader = CG == 1 || rank == 0;
  const int first = static_cast<int>(blockIdx.x) / kCluster;
  const int step = static_cast<int>(gridDim.x) / kCluster;
  const int total = a.n_blocks * a.t_blocks;
  constexpr int kDepth = F::kDepth;
  const int steps = (a.K + 64 * kDepth - 1) / (64 * kDepth);  // stages of the reduction
  const int k0 = S > 1 ? rank * steps / S : 0, k1 = S > 1 ? (rank + 1) * steps / S : steps;
  const int piece = CG == 1 && a.y_fp32 ? kPiece / kDepth : steps;
  const uint32_t stage_tx = kDepth * (kWBytes + a.x_rows * 128);

  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + kStages + s); };
  auto tfull_bar = [&](int b) { return smem_u32(bars + 2 * kStages + b); };
  auto tempty_bar = [&](int b) { return smem_u32(bars + 2 * kStages + 2 + b); };
  const uint32_t group_bar = smem_u32(bars + 2 * kStages + 4);
  const uint32_t red_bar = group_bar + 8;
  const uint32_t drain_bar = red_bar + 8, more_bar = drain_bar + 8;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 8 * CG);  // one arrival per epilogue warp
    }
    mbar_init(group_bar, 8);
    mbar_init(red_bar, 1);
    mbar_init(drain_bar, 1);
    mbar_init(more_bar, 16);  // the epilogue warps of both CTAs
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (S > 1) mbar_arrive_expect_tx(red_bar, F::kRedBytes);
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
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

  if (warp == 0) {
    if (lane == 0) {
      // ---- TMA producer ----
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        int row0, n0;
        tile_at<TN, CG>(a, t, rank, row0, n0);
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
#pragma unroll
              for (int h = 0; h < kDepth; ++h)
                tma_load_2d(st + h * kWBytes, &map_w, full_bar(s), (k * kDepth + h) * 64, n0);
            } else {
              tma_load_2d(st, &map_w, full_bar(s), n0, k * kDepth * 64);
              tma_load_2d(st + kDepth * kWBox, &map_w, full_bar(s), n0 + 64, k * kDepth * 64);
            }
#pragma unroll
            for (int h = 0; h < kDepth; ++h)
              tma_load_2d(st + F::kXOff + h * F::kXBlock, &map_x, full_bar(s), (k * kDepth + h) * 64, row0);
          }
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
      ring_end[0] = static_cast<uint32_t>(s) << 1 | ph;
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---- MMA issuer ----
      constexpr uint32_t idesc = umma_idesc_bf16(128 * CG, TN, !KMAJ);
      int s = 0, buf = 0, par = 0;
      uint32_t ph = 0, acc_ph = 0, more_ph = 0;
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
            for (int kk = 0; kk < 4 * kDepth; ++kk) {
              const uint64_t ad = KMAJ ? umma_desc(st + kk / 4 * kWBytes + kk % 4 * 32)
                                       : umma_desc_mn(st + kk * 16 * 128, kDepth * kWBox);
              const uint64_t bd = umma_desc(st + F::kXOff + kk / 4 * F::kXBlock + kk % 4 * 32);
              if constexpr (CG == 2) umma_bf16_pair(tmem + buf * TN, ad, bd, idesc, k > kp || kk > 0);
              else umma_bf16(tmem + buf * TN, ad, bd, idesc, k > kp || kk > 0);
            }
            issued = true;
            if constexpr (CG == 2) umma_commit_pair(empty_bar(s), 0x3);
            else umma_commit(empty_bar(s));
            if (++s == kStages) { s = 0; ph ^= 1u; }
          }
          if (!ok) break;
          if constexpr (CG == 2) {
            if (a.r <= 32) {  // the ranks of a tile of one adapter
              if (!wait_bounded<true>(more_bar, more_ph, abort_flag, a.dev_status)) { ok = false; break; }
              more_ph ^= 1u;
              umma_fence_after();
              const int* whole = s_whole + par * 8;
              par = par == 2 ? 0 : par + 1;
              bool same = whole[0] >= 0;
              for (int ch = 1; ch < 8; ++ch) same = same && whole[ch] == whole[0];
              if (same) {
                const int rb = a.r <= 16 ? 1 : 2;
                const uint32_t mu = smem_u32(s_more), mt = mu + kMoreU;
                constexpr uint32_t more_idesc = umma_idesc_bf16(128 * CG, TN, true);
                for (int q = 0; q < 2 * rb; ++q)
                  umma_bf16_pair(tmem + buf * TN, umma_desc_mn(mt + q % rb * 2048, 16 * rb * 128),
                                 umma_desc(mu + q * 32), more_idesc, 1);
              }
            }
          }
          if constexpr (CG == 2) umma_commit_pair(tfull_bar(buf), 0x3);
          else umma_commit(tfull_bar(buf));
          if (++buf == 2) { buf = 0; acc_ph ^= 1u; }
        }
      }
      ring_end[1] = issued;
    }
  } else {
    const Epilogue e{s_piece, s_red, s_more, s_id, s_whole, s_starts, abort_flag, tfull_bar(0), tempty_bar(0), group_bar,
                     red_bar, more_bar, tmem, first, step, total, rank, k0, k1, piece};
    if (a.r <= 16) epilogue<TN, S, CG, 1>(a, e, warp, lane);
    else if (a.r <= 32) epilogue<TN, S, CG, 2>(a, e, warp, lane);
    else if (a.r <= 64) epilogue<TN, S, CG, 4>(a, e, warp, lane);
    else epilogue<TN, S, CG, 8>(a, e, warp, lane);
  }

  // ---- teardown ----
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  // No role gives up behind this barrier.  Where one has, whichever it was, MMAs and copies in flight end before
  // the memory that they use is given up.
  if (*abort_flag) {
    if (threadIdx.x == 32 && leader && ring_end[1]) {
      if constexpr (CG == 2) umma_commit_pair(drain_bar, 0x1);
      else umma_commit(drain_bar);
      wait_drain(drain_bar, 0);
    }
    if (threadIdx.x == 0) {
      if (leader) {
        int s = static_cast<int>(ring_end[0] >> 1);
        uint32_t ph = ring_end[0] & 1u;
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
    __syncwarp();
  }
  if constexpr (kCluster > 1) {
    cluster_sync();  // no CTA leaves while a partner may still reach it
    // (after a wait that gave up: nor before the partners' sums that may be on their way)
    if (S > 1 && threadIdx.x == 64 && *abort_flag) wait_drain(red_bar, 0);
  }
  umma_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (CG == 2) umma_dealloc_pair(tmem, F::kTmem);
    else umma_dealloc(tmem, F::kTmem);
  }
  pdl_wait();  // (where the epilogue gave up before its own)
  pdl_trigger();
}

// Clusters of `size` CTAs that can be resident at once, read once per kernel and device.
template <typename Kernel>
int resident_clusters(Kernel kern, int size, int smem, std::mutex& mu, int (&cache)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sm_count() / size * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = sm_count() / size;
    }
    cache[dev] = n;
  }
  return cache[dev];
}

// False, and nothing launched, where S CTAs were to share a tile's reduction and the tiles are
// more than the clusters that are resident at once: a second wave of them takes longer than the
// whole of fewer, longer ones (16 tiles of 7168 x 128, one token: clusters of eight, which do not
// all fit, 18.9 us, of four 14.4, of two 22.7).
template <int TN, int S, int CG, bool KMAJ>
bool launch_project_as(ProjectArgs a, const Operands& o, cudaStream_t s, moe_status& st) {
  using F = Shape<TN, S, CG>;
  auto kern = project_kernel<TN, S, CG, KMAJ>;
  static std::mutex mu;
  static bool done[64] = {};
  st = MOE_ERR_CUDA;
  if (!opt_in(kern, F::kSmem, mu, done)) return true;
  a.n_blocks = static_cast<int>(ceil_div(a.N, 128 * CG));
  a.t_blocks = static_cast<int>(ceil_div(a.seg.T, TN));
  const int64_t tiles = static_cast<int64_t>(a.n_blocks) * a.t_blocks;
  int64_t clusters = std::min<int64_t>(tiles, sm_count());
  if constexpr (S * CG > 1) {
    static std::mutex mu2;
    static int resident[64] = {};
    const int n = resident_clusters(kern, S * CG, F::kSmem, mu2, resident);
    if (n <= 0) return true;
    if (S > 1 && tiles > n) return false;
    clusters = std::min<int64_t>(tiles, n);
  }
  CUtensorMap mw, mx;
  a.x_rows = static_cast<int>(std::min<int64_t>(TN / CG, ceil_div(a.seg.T, 8) * 8));
  // the weight is [K, N] (rows of N), or for the backward [N, K]
  if (!(KMAJ ? map_2d(&mw, o.w, a.N, a.K, a.K, 128) : map_2d(&mw, o.w, a.K, a.N, a.N, 64 * F::kDepth)) ||
      !map_2d(&mx, o.x, a.seg.T, a.K, o.x_stride, a.x_rows))
    return true;
  // Tokens inner: the weight is read once, the rows stay in the L2.  Rows that outgrow it while
  // the weight does not: columns inner.
  constexpr int64_t kL2Budget = 80ll << 20;
  a.n_inner = static_cast<int64_t>(a.seg.T) * a.K * 2 > kL2Budget &&
              static_cast<int64_t>(a.N) * a.K * 2 <= kL2Budget;
  launch_clustered(kern, dim3(static_cast<unsigned>(clusters * S * CG)), kThreads, F::kSmem, S * CG, s,
                   mw, mx, a);
  st = launch_status();
  return true;
}

template <int TN, bool KMAJ>
moe_status launch_flat(const ProjectArgs& a, const Operands& o, int split, cudaStream_t s) {
  moe_status st = MOE_ERR_CUDA;
  switch (split) {
    case 4:
      if (launch_project_as<TN, 4, 1, KMAJ>(a, o, s, st)) return st;
      [[fallthrough]];
    case 2:
      if (launch_project_as<TN, 2, 1, KMAJ>(a, o, s, st)) return st;
      [[fallthrough]];
    default: launch_project_as<TN, 1, 1, KMAJ>(a, o, s, st); return st;
  }
}

}  // namespace
}  // namespace adapter
}  // namespace moe
