// Projections with 4-bit weights: y[r][n] = sum_k x[r][k] w[n][k],
// w[n][k] = code[n][k] * scale[n][k / group], for few rows of x
// (up to 8 of fp32, 16 of bf16; gdn_quant_wide.cu has the form for more).
//
// Bound by reading the weights (half a byte each); the arithmetic runs on
// mma.sync m16n8k16 so that it stays below that: A is 16 weight rows (codes as
// 16-bit floats, exact), B the rows of x, and the fp32 products of one group
// are multiplied by the group's scale and added up in fp32.
// (A tcgen05 product puts the codes through shared memory first, and its
// 128-row tiles leave too few of them to split over the SMs; a handful of
// columns does not pay for that.)
//
//   fp32 x   two columns per row: x 2^e = hi + lo in fp16 (22 bits; e by row
//            and block of 256, so that the largest element is in [2^14, 2^15);
//            elements below 2^-17 of it keep fewer, the lo part ends at 2^-24)
//   bf16 x   one column per row, as it is; the codes as bf16
//
// Weights.  A warp takes blocks of 16 rows x 256 codes (128 bytes of each row)
// through a ring of its own in shared memory: asynchronous 16-byte copies, 8
// lanes to a row, so that a request is four whole lines (fragment-shaped loads,
// 64 bytes of 8 rows, spent more cycles on cache tags than the arithmetic
// takes), chunks XOR-ed by the row.  ldmatrix hands lane (row g, t) word t of a
// row's 16-byte chunk, 8 codes; chunk i is k 32 i .. 32 i + 31, so every product
// step stays inside one group whatever the group size.  The sum over k may run
// in any order: the codes are used as they unpack (elements 0 and 4 of a word
// are one register, 1 and 5 the next, ...), and x is put into shared memory in
// that order.
//
// Work split.  One CTA of 16 warps per SM; a CTA, or a cluster
// of up to 8 that cut K between them (few tiles, or much x to convert), takes a
// range of 16-row tiles.  Inside a CTA the (tile, block) pairs are one list, cut
// evenly over the warps whatever the sizes.  At the end of a tile, or of its
// share, a warp stores its partial sums in a slot of its own in the CTA that
// adds up the tile; slots are added in a fixed order, so results are the same
// bits on every call.
//
// One row against 10240 x 5120, weights from HBM (15 of them in turn, calls back
// to back): 11.5 us (27 MB, 2.4 TB/s), 8 rows of fp32 15.6, of bf16 14.9, 16 rows of
// bf16 19.0; a single call behind a flushed L2 14.6 (one row), 18.7 (8 of fp32).
// 48 x 5120 (a layer's gates) 4.9 us.  What is left is a start of 2 us, the x that every CTA converts,
// the products' issue (the SIMD lanes unpack 8 codes in 14 instructions) and for
// clusters two barriers.

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <array>
#include <map>
#include <mutex>
#include <type_traits>

#include "gdn_internal.cuh"
#include "gdn_vec.cuh"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kBlock = 256;   // k elements of a block
constexpr int kTile = 16;     // weight rows of a tile
constexpr int kBlockBytes = kTile * kBlock / 2;
constexpr int kXBlock = kBlock * 2;  // bytes of a block of a column of x
constexpr int kDepth = 3;  // blocks of a warp's ring
constexpr int kSmemMax = 220 * 1024;
// Costs of make_plan(), relative to a block.
constexpr double kXCost = 0.1, kClusterCost[4] = {0.0, 5.0, 8.0, 20.0};

struct QuantArgs {
  const void *x;
  const uint8_t *qw;
  const __half *sc;
  void *y;
  int rows, N, K;
  int tiles, blocks;      // 16-row tiles, 256-element blocks of a row
  int round_tiles;        // tiles of a cluster in one round
  int round_blocks;       // blocks of a CTA's slice in one round
  int csize, slots;       // CTAs of a cluster, slots of partial sums
  int columns;            // of x in shared memory (those beyond are not used)
  int sc_shared;          // the round's scales are copied to shared memory
};

// Blocks of CTA `rank`'s slice of a round: an even share where one round takes
// all of K, else round_blocks in every round (behind the end of K they are
// zeros), so that a warp's share of tiles is the same in all rounds.
__device__ __forceinline__ void slice(const QuantArgs &P, int csize, int rank, int &lo, int &n) {
  if (P.blocks <= csize * P.round_blocks) {
    lo = (unsigned)(P.blocks * rank) / (unsigned)csize;
    n = (unsigned)(P.blocks * (rank + 1)) / (unsigned)csize - lo;
  } else {
    lo = rank * P.round_blocks;
    n = P.round_blocks;
  }
}

// The most warps that share a tile, of nt tiles and at most `blocks` blocks.
__host__ __device__ inline int most_warps(int nt, int blocks) {
  int m = (kWarps + nt - 1) / nt + 1;
  if (m > blocks) m = blocks;
  return m < kWarps ? m : kWarps;
}

// Warp w's share [share(w), share(w + 1)) of a list of `total` pairs.
__device__ __forceinline__ int share(unsigned total, int w) {
  return (int)((unsigned long long)total * w / kWarps);
}

// 8 codes of a word as four registers of two 16-bit floats: elements (0, 4),
// (1, 5), (2, 6), (3, 7).  A code c is stored as c + 16 (c < 0); flipping its
// bit 3 gives c + 8, which as the low mantissa bits of 1024 (fp16) or 128
// (bf16) is 1032 + c or 136 + c.  (The 136 left in, and a group's product started
// at -136 sum x, was no faster and left rounding errors of a sum of |x| where
// the codes are zeros.)
template <bool kBf16>
__device__ __forceinline__ void codes(uint32_t u, uint32_t (&r)[4]) {
  if (kBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = ((u >> (4 * i)) & 0x000f000fu) ^ 0x43084308u;
      const __nv_bfloat162 d = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                       __floats2bfloat162_rn(-136.f, -136.f));
      r[i] = *reinterpret_cast<const uint32_t *>(&d);
    }
  } else {
    const __half2 m = __floats2half2_rn(-1032.f, -1032.f);
    const __half2 s = __floats2half2_rn(0.0625f, 0.0625f), m16 = __floats2half2_rn(-72.f, -72.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = u >> (8 * i);
      const uint32_t a = (v & 0x000f000fu) ^ 0x64086408u;   // 1032 + c
      const uint32_t b = (v & 0x00f000f0u) ^ 0x64806480u;   // 1024 + 16 (8 + c)
      const __half2 da = __hadd2(*reinterpret_cast<const __half2 *>(&a), m);
      const __half2 db = __hfma2(*reinterpret_cast<const __half2 *>(&b), s, m16);
      r[2 * i] = *reinterpret_cast<const uint32_t *>(&da);
      r[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&db);
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1,
                                    const float (&c)[4]) {
  if (kBf16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  // (bytes < 16: the rest is filled with zeros and not read)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Four 8 x 16-byte matrices; lane l gives the address of row l & 7 of matrix
// l >> 3 and receives word l & 3 of row l >> 2 of each.
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool kBf16, int kNT, int kGroup>
__global__ void __launch_bounds__(kThreads, 1)
    quant_linear_kernel(const QuantArgs P) {
  using T = typename std::conditional<kBf16, __nv_bfloat16, float>::type;
  constexpr int kCols = 8 * kNT;
  constexpr int kRowsX = kBf16 ? kCols : kCols / 2;  // rows of x of a pass
  constexpr int kSc = kBlock / kGroup;               // scales of a block
  constexpr int kSums = kBf16 ? 4 : 2;               // of a lane and m16n8 tile
  extern __shared__ __align__(16) unsigned char smem[];
  const cg::cluster_group cl = cg::this_cluster();
  const int csize = P.csize, crank = csize > 1 ? (int)cl.block_rank() : 0;
  const int cluster = (unsigned)blockIdx.x / (unsigned)csize;
  const int clusters = (unsigned)gridDim.x / (unsigned)csize;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  const int gr = lane >> 2, t = lane & 3;

  // shared memory: the warps' rings, partial sums, x (a column is round_blocks *
  // 512 + 64 bytes), then by block: 2^-e of each row (fp32), then by slice and
  // tile: the first warp in it and the number of warps, then the scales of the
  // round's rows
  const uint32_t xstride = (uint32_t)P.round_blocks * kXBlock + 64;
  const uint32_t ring =
      (uint32_t)__cvta_generic_to_shared(smem) + warp * kDepth * kBlockBytes;
  float *slots = reinterpret_cast<float *>(smem + kWarps * kDepth * kBlockBytes);
  unsigned char *xs =
      reinterpret_cast<unsigned char *>(slots) + (size_t)P.slots * kTile * kRowsX * 4;
  float *side = reinterpret_cast<float *>(xs + (size_t)P.columns * xstride);
  unsigned char *tab = reinterpret_cast<unsigned char *>(
      side + (kBf16 ? 0 : P.round_blocks * kRowsX));
  __half *scs = reinterpret_cast<__half *>(
      smem + (((size_t)(tab - smem) + 2 * csize * P.round_tiles + 15) & ~(size_t)15));
  // this lane's column of x in each n8 tile (columns that are not there: any)
  const unsigned char *xl[kNT];
#pragma unroll
  for (int j = 0; j < kNT; ++j)
    xl[j] = xs + (8 * j + gr < P.columns ? 8 * j + gr : 0) * xstride + t * 16;

  // behind the kernel before it: nothing is read or written before it has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (csize > 1) cl.sync();  // every CTA's shared memory is there

  const size_t wrow = (size_t)P.K / 2;
  const int groups = P.K / kGroup;

  const int nr = P.rows;  // at most kRowsX
  for (int t0 = cluster * P.round_tiles; t0 < P.tiles; t0 += clusters * P.round_tiles) {
    const int nt = min(P.round_tiles, P.tiles - t0);
    const int own = (unsigned)(nt + csize - 1) / (unsigned)csize;  // tiles a CTA adds up
    const int most = most_warps(nt, P.round_blocks);
    for (int kr = 0; kr < P.blocks; kr += csize * P.round_blocks) {
      int b_lo, nb;
      slice(P, csize, crank, b_lo, nb);
      b_lo += kr;
      const unsigned total = nt * nb;
      int pos = share(total, warp);
      const int end = share(total, warp + 1);

      // ---- weights: the next block of this warp's list into its ring.  Lane
      // l copies 16-byte chunk l & 7 of rows (l >> 3) + 4 i; rows and chunks
      // behind the end are zeros.
      const int crow = lane >> 3, chunk = lane & 7;
      const uint32_t step = 4 * (uint32_t)wrow;  // four rows
      // (row & 7 of rows crow + 4 i alternates between two values)
      const uint32_t d0 = ring + crow * 128 + ((chunk ^ crow) << 4);
      const uint32_t d1 = ring + (crow + 4) * 128 + ((chunk ^ (crow + 4)) << 4);
      int lpos = pos, lb = 0, lt = 0;
      uint32_t ld = 0;
      const uint8_t *wp = nullptr;
      int left = 0;  // rows of the tile from crow on
      auto aim = [&]() {
        const int n0 = (t0 + lt) * kTile + crow;
        left = P.N - n0;
        wp = P.qw + (size_t)min(n0, P.N - 1) * wrow + (size_t)(b_lo + lb) * (kBlock / 2) +
             16 * chunk;
      };
      if (pos < end) {
        lt = (unsigned)pos / (unsigned)nb;
        lb = pos - lt * nb;
        aim();
      }
      auto fetch = [&]() {
        if (lpos < end) {
          if ((t0 + lt + 1) * kTile <= P.N && (b_lo + lb + 1) * kBlock <= P.K) {
            cp_async16(d0 + ld, wp, 16);
            cp_async16(d1 + ld, wp + step, 16);
            cp_async16(d0 + ld + 1024, wp + 2 * step, 16);
            cp_async16(d1 + ld + 1024, wp + 3 * step, 16);
          } else {
            const int in = (b_lo + lb) * kBlock + 32 * chunk < P.K ? 16 : 0;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int bytes = 4 * i < left ? in : 0;
              cp_async16((i & 1 ? d1 : d0) + ld + 1024 * (i >> 1), bytes ? wp + i * step : P.qw,
                         bytes);
            }
          }
          if (++lb == nb) {
            lb = 0;
            ++lt;
            aim();
          } else {
            wp += kBlock / 2;
          }
          ++lpos;
          ld = ld == (kDepth - 1) * kBlockBytes ? 0 : ld + kBlockBytes;
        }
        cp_async_commit();
      };
      // ---- the scales of the round's rows (contiguous), once a round
      if (P.sc_shared && !kr) {
        const int n0 = t0 * kTile, nrows = min(nt * kTile, P.N - n0);
        const int bytes = nrows * groups * 2;
        const unsigned char *src = reinterpret_cast<const unsigned char *>(P.sc + (size_t)n0 * groups);
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(scs);
        for (int e = tid * 16; e < bytes; e += kThreads * 16)
          cp_async16(dst + e, src + e, min(16, bytes - e));
      }
      cp_async_commit();

      // ---- x: this slice of the rows in the order of use; half a warp to
      // 128 elements of a row.  The first part is read before the weights
      // are asked for.
      if (kr || t0 != cluster * P.round_tiles) __syncthreads();  // readers are done
      {
        const int p = lane & 15, halves = 2 * nb;
        int b = 2 * warp + (lane >> 4), r = 0;
        auto wrap = [&]() {
          while (b >= halves && r < kRowsX) {
            b -= halves;
            ++r;
          }
        };
        wrap();
        struct Part {
          float v[8];
        };
        auto read = [&]() {
          Part x = {};
          const int k = b_lo * kBlock + b * 128 + 8 * p;
          if (r < nr && k < P.K) load8(static_cast<const T *>(P.x) + (size_t)r * P.K + k, x.v);
          return x;
        };
        // (both halves run the same number of turns: shuffles inside)
        const int turns = (nr * halves + 2 * kWarps - 1) / (2 * kWarps);
        Part x = read();
        for (int turn = 0; turn < turns || turn == 0; ++turn) {
          const int cb = b, cr = r;
          const Part c = x;
          if (turn == 0) {
            // The weights are asked for once the first part of x is here: a
            // burst of weights from every SM would keep it waiting for twice
            // the time.
            asm volatile("" ::"f"(c.v[0]) : "memory");
#pragma unroll
            for (int d = 0; d < kDepth - 1; ++d) fetch();
          }
          b += 2 * kWarps;
          wrap();
          if (turn + 1 < turns) x = read();
          unsigned char *dst = xs + cb * (kXBlock / 2) + p * 16;
          if (kBf16) {
            if (cr < nr) {
              // elements (0, 4), (1, 5), (2, 6), (3, 7)
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                o[j] = __byte_perm(__float_as_uint(c.v[j]), __float_as_uint(c.v[j + 4]), 0x7632);
              *reinterpret_cast<uint4 *>(dst + cr * xstride) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else {
            int m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_int(c.v[i]) & 0x7fffffff);
            // (the other half warp has the other half of the same block)
#pragma unroll
            for (int d = 16; d; d >>= 1) m = max(m, __shfl_xor_sync(kFull, m, d));
            // 2^e: the block's largest element into [2^14, 2^15)
            const int ex = min(141 - (m >> 23), 126);
            const float f = __int_as_float((ex + 127) << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x0 = c.v[i] * f, x1 = c.v[i + 4] * f;
              const __half2 h = __floats2half2_rn(x0, x1);
              const float2 g = __half22float2(h);
              const __half2 l = __floats2half2_rn(x0 - g.x, x1 - g.y);
              hi[i] = *reinterpret_cast<const uint32_t *>(&h);
              lo[i] = *reinterpret_cast<const uint32_t *>(&l);
            }
            if (cr < nr) {
              dst += 2 * cr * xstride;
              *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4 *>(dst + xstride) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
              if (lane == 0) side[(cb >> 1) * kRowsX + cr] = __int_as_float((127 - ex) << 23);
            }
          }
        }
      }
      // the warps in each tile of each slice: share(w) <= i exactly for
      // w <= (kWarps (i + 1) - 1) / total (lists shorter than the warps: one
      // pair each, numbered by block)
      if (!kr)
        for (int e = tid; e < csize * nt; e += kThreads) {
          const int q = (unsigned)e / (unsigned)nt, tile = e - q * nt;
          int q_lo, qb;
          slice(P, csize, q, q_lo, qb);
          const unsigned all = nt * qb;
          int w_lo = 0, n = qb;
          if (all >= kWarps) {
            w_lo = (kWarps * (tile * qb + 1) - 1) / all;
            n = (kWarps * (tile + 1) * qb - 1) / all - w_lo + 1;
          }
          tab[2 * e] = (unsigned char)w_lo;
          tab[2 * e + 1] = (unsigned char)n;
        }
      cp_async_wait<kDepth - 1>();  // (the scales)
      __syncthreads();

      // ---- products
      float acc[kNT][kSums];
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int i = 0; i < kSums; ++i) acc[j][i] = 0.f;
      int tile = 0, blk = 0;
      uint32_t rd = 0;
      if (pos < end) {
        tile = (unsigned)pos / (unsigned)nb;
        blk = pos - tile * nb;
      }
      // this lane's ldmatrix row: row lane & 7, chunk lane >> 3 (then + 4, and
      // rows + 8)
      const uint32_t lrow = (lane & 7) * 128;
      const uint32_t lc0 = lrow + ((((uint32_t)lane >> 3) ^ (lane & 7)) << 4);
      const uint32_t lc1 = lrow + (((((uint32_t)lane >> 3) + 4) ^ (lane & 7)) << 4);
      const __half *s0p = nullptr, *s1p = nullptr;
      auto scales_of = [&]() {  // (rows behind the last one: its scales)
        const int n0 = t0 * kTile, last = P.N - 1 - n0;
        const __half *sc = P.sc_shared ? scs : P.sc + (size_t)n0 * groups;
        s0p = sc + (size_t)min(tile * kTile + gr, last) * groups;
        s1p = sc + (size_t)min(tile * kTile + gr + 8, last) * groups;
      };
      if (pos < end) scales_of();
      for (; pos < end; ++pos) {
        cp_async_wait<kDepth - 2>();
        __syncwarp();  // every lane's copies of this block have landed
        const uint32_t st = ring + rd;
        rd = rd == (kDepth - 1) * kBlockBytes ? 0 : rd + kBlockBytes;
        uint32_t w0[8], w1[8];  // rows gr, gr + 8: chunks 0..7
        {
          uint32_t a[4], b[4], c[4], d[4];
          ldmatrix4(st + lc0, a);
          ldmatrix4(st + lc1, b);
          ldmatrix4(st + 1024 + lc0, c);
          ldmatrix4(st + 1024 + lc1, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w0[i] = a[i];
            w0[i + 4] = b[i];
            w1[i] = c[i];
            w1[i + 4] = d[i];
          }
        }
        // (the slot that is filled now was read a turn ago, and every lane
        // has passed the barrier above since)
        fetch();
        float part[kNT][4], un[kNT];
        if (!kBf16)
#pragma unroll
          for (int j = 0; j < kNT; ++j) un[j] = side[blk * kRowsX + 4 * j + t];
        const int g0 = (b_lo + blk) * kSc;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          constexpr int kSteps = kGroup / 32;
          const int g = i / kSteps;
          if (i % kSteps == 0) {
#pragma unroll
            for (int j = 0; j < kNT; ++j)
#pragma unroll
              for (int c = 0; c < 4; ++c) part[j][c] = 0.f;
          }
          uint32_t c0[4], c1[4];
          codes<kBf16>(w0[i], c0);
          codes<kBf16>(w1[i], c1);
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            const uint4 x4 = *reinterpret_cast<const uint4 *>(xl[j] + blk * kXBlock + i * 64);
            mma<kBf16>(part[j], c0[0], c1[0], c0[1], c1[1], x4.x, x4.y, part[j]);
            mma<kBf16>(part[j], c0[2], c1[2], c0[3], c1[3], x4.z, x4.w, part[j]);
          }
          if ((i + 1) % kSteps == 0) {
            // (a group behind the last one counts as 0 against any scale)
            const int gi = min(g0 + g, groups - 1);
            const float f0 = g0 + g < groups ? __half2float(s0p[gi]) : 0.f;
            const float f1 = g0 + g < groups ? __half2float(s1p[gi]) : 0.f;
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
              if (kBf16) {
                acc[j][0] = fmaf(f0, part[j][0], acc[j][0]);
                acc[j][1] = fmaf(f0, part[j][1], acc[j][1]);
                acc[j][2 % kSums] = fmaf(f1, part[j][2], acc[j][2 % kSums]);
                acc[j][3 % kSums] = fmaf(f1, part[j][3], acc[j][3 % kSums]);
              } else {  // the hi and lo columns of one row
                acc[j][0] = fmaf(f0 * un[j], part[j][0] + part[j][1], acc[j][0]);
                acc[j][1] = fmaf(f1 * un[j], part[j][2] + part[j][3], acc[j][1]);
              }
            }
          }
        }
        ++blk;
        if (blk == nb || pos + 1 == end) {
          // partial sums of the tile, to their slot in the CTA that adds it
          // up: [slice][tile][warp in the tile]
          const int at = (unsigned)tile / (unsigned)csize, to = tile - at * csize;
          const int nth = total < kWarps ? blk - 1 : warp - tab[2 * (crank * nt + tile)];
          float *sl = slots + (size_t)((crank * own + at) * most + nth) * kTile * kRowsX +
                      gr * kRowsX;
          if (csize > 1) sl = cl.map_shared_rank(sl, to);
#pragma unroll
          for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int i = 0; i < kSums; ++i) {
              // bf16: rows gr, gr + 8 and columns 2 t, 2 t + 1; fp32: the two
              // rows of x row t
              const int row = 8 * (kBf16 ? i >> 1 : i);
              const int col = kBf16 ? 8 * j + 2 * t + (i & 1) : 4 * j + t;
              if (col < nr) {
                float v = acc[j][i];
                if (kr) v += sl[row * kRowsX + col];
                sl[row * kRowsX + col] = v;
              }
              acc[j][i] = 0.f;
            }
          blk = 0;
          ++tile;
          if (pos + 1 < end) scales_of();
        }
      }
      cp_async_wait<0>();
    }

    // ---- the sum over slices and warps, tiles crank, crank + csize, ...
    if (csize > 1)
      cl.sync();
    else
      __syncthreads();
    for (int e = tid; e < own * kTile * nr; e += kThreads) {
      const int r = (unsigned)e / (unsigned)(own * kTile), c = e - r * own * kTile;
      const int at = c / kTile, tile = at * csize + crank, n = (t0 + tile) * kTile + c % kTile;
      if (tile >= nt || n >= P.N) continue;
      float sum = 0.f;
      for (int q = 0; q < csize; ++q) {
        const float *sl = slots + ((size_t)((q * own + at) * most) * kTile + c % kTile) * kRowsX + r;
        const int cnt = tab[2 * (q * nt + tile) + 1];
        for (int w = 0; w < cnt; ++w, sl += kTile * kRowsX) sum += *sl;
      }
      const size_t out = (size_t)r * P.N + n;
      if (kBf16)
        static_cast<__nv_bfloat16 *>(P.y)[out] = __float2bfloat16_rn(sum);
      else
        static_cast<float *>(P.y)[out] = sum;
    }
    // the slots are read
    if (csize > 1 && t0 + clusters * P.round_tiles < P.tiles) cl.sync();
  }
}

struct Plan {
  int nt, csize, clusters, round_tiles, round_blocks, slots, columns, sc_shared;
  size_t smem;
};

// Cluster size and rounds for the shape.  The cost of a CTA, in blocks: its
// list, its share of x, and for a cluster its two barriers.
// `most`: clusters of 1, 2, 4, 8 CTAs that the GPU runs at once.
Plan make_plan(int rows, int N, int K, int group, bool bf16, const int (&most)[4]) {
  Plan p = {};
  const int cols = bf16 ? rows : 2 * rows;
  p.nt = cols <= 8 ? 1 : 2;
  p.columns = cols;
  const int rows_x = bf16 ? 8 * p.nt : 4 * p.nt;
  const int tiles = (N + kTile - 1) / kTile, blocks = (K + kBlock - 1) / kBlock;
  const int groups = K / group;
  // shared memory of cluster size c, rt tiles and rb blocks a round; the
  // scales where they fit
  auto bytes = [&](int c, int rt, int rb) {
    const int last = tiles % rt;  // tiles of the last round, if fewer
    const auto slots = [&](int n) {
      return n ? c * ((n + c - 1) / c) * most_warps(n, rb) : 0;
    };
    p.slots = slots(rt) > slots(last) ? slots(rt) : slots(last);
    const size_t need = (size_t)kWarps * kDepth * kBlockBytes +
                        (size_t)p.slots * kTile * rows_x * 4 +
                        (size_t)p.columns * ((size_t)rb * kXBlock + 64) +
                        (bf16 ? 0 : (size_t)rb * 4 * rows_x) +
                        (((size_t)2 * c * rt + 31) & ~(size_t)15);
    const size_t sc = (((size_t)rt * kTile * groups * 2) + 15) & ~(size_t)15;
    p.sc_shared = need + sc <= kSmemMax;
    return need + (p.sc_shared ? sc : 0);
  };
  double best = 1e300;
  for (int i = 0; i < 4; ++i) {
    const int c = 1 << i, clusters = most[i] < tiles ? most[i] : tiles;
    const int rt = (tiles + clusters - 1) / clusters, rb = (blocks + c - 1) / c;
    double cost = (double)rt * rb + kXCost * rows * rb + kClusterCost[i];
    if (bytes(c, rt, rb) > kSmemMax) cost += 1e100;  // in rounds: the largest cluster
    if (cost < best || (cost >= 1e100 && best >= 1e100)) {
      best = cost;
      p.csize = c;
      p.clusters = (tiles + rt - 1) / rt;
      p.round_tiles = rt;
      p.round_blocks = rb;
    }
  }
  // Rounds where shared memory does not hold a CTA's share: at least 8 tiles
  // at a time, then as many blocks as fit (one block of 8 tiles always does).
  while (p.round_tiles > 8 && bytes(p.csize, p.round_tiles, p.round_blocks) > kSmemMax)
    p.round_tiles = (p.round_tiles + 1) / 2;
  while (p.round_blocks > 1 && bytes(p.csize, p.round_tiles, p.round_blocks) > kSmemMax)
    p.round_blocks = (p.round_blocks + 1) / 2;
  p.smem = bytes(p.csize, p.round_tiles, p.round_blocks);
  return p;
}

template <bool kBf16, int kNT, int kGroup>
cudaError_t launch(const QuantArgs &a, const Plan &p, cudaStream_t stream) {
  const auto kernel = quant_linear_kernel<kBf16, kNT, kGroup>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.clusters * p.csize));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.csize;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (p.csize == 1) {
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// How many clusters of 1, 2, 4, 8 such CTAs (one per SM) the current device runs
// at once: GPCs differ in their SMs, so clusters of 8 leave some of them idle
// (15 of the 19 that 152 SMs would hold on a GB300).  Asked once per device.
cudaError_t cluster_counts(int (&most)[4]) {
  static std::mutex lock;
  static std::map<int, std::array<int, 4>> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> hold(lock);
  auto it = known.find(dev);
  if (it == known.end()) {
    const auto kernel = quant_linear_kernel<true, 1, 128>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    std::array<int, 4> n;
    for (int i = 0; i < 4; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(8);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kSmemMax;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 1u << i;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n[i], kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (n[i] < 1) n[i] = 1;
    }
    it = known.emplace(dev, n).first;
  }
  for (int i = 0; i < 4; ++i) most[i] = it->second[i];
  return cudaSuccess;
}

template <bool kBf16, int kNT>
cudaError_t by_group(int group, const QuantArgs &a, const Plan &p, cudaStream_t stream) {
  return group == 128  ? launch<kBf16, kNT, 128>(a, p, stream)
         : group == 64 ? launch<kBf16, kNT, 64>(a, p, stream)
                       : launch<kBf16, kNT, 32>(a, p, stream);
}

template <bool kBf16>
cudaError_t by_columns(int group, const QuantArgs &a, const Plan &p, cudaStream_t stream) {
  return p.nt == 1 ? by_group<kBf16, 1>(group, a, p, stream)
                   : by_group<kBf16, 2>(group, a, p, stream);
}

}  // namespace

cudaError_t launch_quant_linear(const void *x, const unsigned char *qw,
                                const void *scales, void *y, int rows, int N,
                                int K, int group, bool bf16,
                                cudaStream_t stream) {
  if (rows == 0 || N == 0) return cudaSuccess;
  // More than 16 columns go to products of 128 weight rows: 64 rows of bf16
  // against 5120 x 6144 took 54 us here, 32 columns at a time, and take 18.9
  // there; 16 rows take 14 us here (17 there).
  if ((bf16 ? rows : 2 * rows) > 16)
    return launch_quant_linear_wide(x, qw, scales, y, rows, N, K, group, bf16, stream);
  int most[4];
  const cudaError_t e = cluster_counts(most);
  if (e != cudaSuccess) return e;
  const Plan p = make_plan(rows, N, K, group, bf16, most);
  const QuantArgs a{x, qw, static_cast<const __half *>(scales), y, rows, N, K,
                    (N + kTile - 1) / kTile, (K + kBlock - 1) / kBlock, p.round_tiles, p.round_blocks,
                    p.csize, p.slots, p.columns, p.sc_shared};
  return bf16 ? by_columns<true>(group, a, p, stream) : by_columns<false>(group, a, p, stream);
}

}  // namespace gdn
