// Attention of new tokens over a paged key-value cache, for sm_103a
// (gdn_attn_step_m): the kernel, compiled for one head size by each of
// gdn_attn_64.cu, gdn_attn_128.cu and gdn_attn_256.cu.
//
// What it computes (sequence b, key head h, row r = (token m, query head of
// h's group)):
//     s_j = scale q_r . k_j,  j <= start[b] + m;
//     o_r = sum_j e^{s_j} v_j / sum_j e^{s_j}.
// One pass over the cache: each warp keeps the reference m_r (a running
// maximum), the sum l_r and the sums over v of its rows, and all are
// rescaled when the maximum grows.  Parts of a sequence meet by
//     l = sum_p l_p 2^{m_p - m},  o = sum_p acc_p 2^{m_p - m} / l.
//
// Work split.  A sequence's positions are cut into chunks of kWarps x kTT, a
// tile of kTT positions for each warp; chunks of all (sequence, head, row tile)
// items follow one another and every CTA takes an equal, contiguous share of
// that list, found from the lengths on the device.  An item that lies within one
// CTA is finished there; of the others a CTA leaves at most two parts in the
// workspace, which attn_join_kernel adds in order.  So the workspace does not
// grow with the batch, ragged batches fill the GPU, and the same lengths give
// the same bits.
//
// Loads.  Each warp copies its own tiles, K and V in turn, 16 bytes a lane
// (cp.async) into its own ring: no barrier within an item, and the copies of the
// next item are under way while this one is joined.  The rings hold about 100 KB
// an SM in flight.  16-byte units are stored permuted, so that the reads below
// meet no bank twice.
//
// Products.  A tile of 16 rows by mma.sync m16n8k16 with fp32 sums; the work is
// bound by the copies, not by the products (8 rows of 8-bit codes: 16
// multiply-adds a byte).  The channels of a product may come in any order as
// long as q follows, so a lane reads 16 bytes of a K row and has 4 (bf16: 2)
// products' worth of operands.
//   8 bits   codes are exact in fp16; q of a row is scaled by a power of two to
//            below 2^14 and cut into fp16 parts (bf16: one, exact for elements
//            above 2^-28 of the row's largest; fp32: two, 22 bits); scales are
//            applied to the scores, and to the weights: w_j = p_j vscale_j.  The
//            reference follows s_j + log2 vscale_j, so that w is at most 2^15 and
//            the largest is at least 1, and w is cut into two fp16 parts (22 bits,
//            2^-37 of the largest).
//   bf16     q one bf16 part or (fp32) three, weights two parts (16 bits) or
//            (fp32) three.
// Up to 8 rows: the parts lie in the two halves of the 16-row tile, so that the
// second part costs no second product; more rows: one product for each part.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "gdn_internal.cuh"

namespace gdn {
namespace attn {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr float kNone = -1e30f;  // the reference of rows that have seen nothing
constexpr float kSlack = 3.0f;   // how far the maximum may pass it (log2)
constexpr int kSms = 152;

// Sizes of a variant.
template <int kHd, int kKind>
struct Sizes {
  static constexpr int kBytes = kKind == kKvBf16 ? 2 : 1;
  static constexpr int kRow = kHd * kBytes;                   // bytes of a row
  static constexpr int kTT = kBytes == 1 || kRow <= 128 ? 32 : 16;  // positions of a tile
  static constexpr int kUnit = kTT * kRow;                    // K or V of a tile
  static constexpr int kSlot = kUnit + (kKind == kKvBf16 ? 0 : 8 * kTT);  // and scales
  static constexpr int kCtas = kHd == 256 ? 1 : 2;            // CTAs an SM
  static constexpr int kRing = (kCtas == 1 ? 26 : 13) * 1024;  // a warp's ring
  static constexpr int kSlots = kRing / kSlot;
  static constexpr int kChunk = kWarps * kTT;
};

// Rows of an item: 8 (R = 1) or 16 (R = 2).
template <int kKind, bool kBf16>
struct Parts {
  static constexpr int kQ = kKind == kKvBf16 ? (kBf16 ? 1 : 3) : (kBf16 ? 1 : 2);
  static constexpr int kP = kKind == kKvBf16 ? (kBf16 ? 2 : 3) : 2;
};
__host__ __device__ constexpr int tiles_of(int parts, int R) { return R == 1 ? (parts + 1) / 2 : parts; }

// A CTA's share of the chunks, and where an item's parts lie.
struct Share {
  long long total;
  int ctas;
  __host__ __device__ long long first(int cta) const { return total * cta / ctas; }
  __host__ __device__ int of(long long unit) const {
    return (int)(((unit + 1) * ctas - 1) / total);
  }
};

// Positions that a sequence's new tokens see, and its first new one; 0 where
// there is nothing to do.
__device__ __forceinline__ int length_of(const AttnArgs &P, int b, int &start) {
  start = P.start[b];
  const int n = P.counts ? P.counts[b] : P.M;
  const long long room = (long long)P.cols << P.c.page_shift;
  if (n <= 0 || n > P.M || start < 0 || (long long)start + n > room) return 0;
  return start + n;
}

__device__ __forceinline__ void cp16(uint32_t to, const void *from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void wait_for() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(s));
  return r;
}

// c += a b: 16 rows, 8 columns, 16 channels; fp16 or bf16.
template <bool kHalf>
__device__ __forceinline__ void mma(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  if (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Four codes as two pairs of fp16.
template <int kKind>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (kKind == kKvInt8) {
    // u = code + 128 behind the bits of 1024, which is 1024 + u; less 1152
    w ^= 0x80808080u;
    lo = prmt(w, 0x64646464u, 0x4140);
    hi = prmt(w, 0x64646464u, 0x4342);
    const __half2 off = __half2(__half_raw{0x6480}, __half_raw{0x6480});
    __half2 a = __hsub2(*reinterpret_cast<__half2 *>(&lo), off);
    __half2 b = __hsub2(*reinterpret_cast<__half2 *>(&hi), off);
    lo = *reinterpret_cast<uint32_t *>(&a);
    hi = *reinterpret_cast<uint32_t *>(&b);
  } else {
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// Two numbers as pairs of 16-bit parts: p[0] the nearest, p[i] of what is left.
template <bool kHalf, int kN>
__device__ __forceinline__ void cut(float x, float y, uint32_t (&p)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if (kHalf) {
      const __half2 h = __floats2half2_rn(x, y);
      p[i] = *reinterpret_cast<const uint32_t *>(&h);
      if (i + 1 < kN) {
        x -= __low2float(h);
        y -= __high2float(h);
      }
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
      p[i] = *reinterpret_cast<const uint32_t *>(&h);
      if (i + 1 < kN) {
        x -= __uint_as_float(p[i] << 16);
        y -= __uint_as_float(p[i] & 0xffff0000u);
      }
    }
  }
}

// log2 of a scale to about 0.1, from its bits, between -90 and 129.
__device__ __forceinline__ float rough_log2(float s) {
  return fmaxf(fmaf((float)__float_as_int(s), 0x1p-23f, -127.0f), -90.0f);
}

__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  x[0] = __uint_as_float(u.x << 16);
  x[1] = __uint_as_float(u.x & 0xffff0000u);
  x[2] = __uint_as_float(u.y << 16);
  x[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float *p, const float (&x)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]);
  const __nv_bfloat162 b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                             *reinterpret_cast<const uint32_t *>(&b));
}

// Sum over the block of two counts.
__device__ __forceinline__ void block_sums(long long &x, long long &y, long long *room) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    x += __shfl_xor_sync(kFull, x, d);
    y += __shfl_xor_sync(kFull, y, d);
  }
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    room[warp] = x;
    room[kWarps + warp] = y;
  }
  __syncthreads();
  x = y = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    x += room[w];
    y += room[kWarps + w];
  }
}

// Where a 16-byte unit of a row lies in a tile (see the reads).
template <int kRow>
__device__ __forceinline__ int k_place(int r, int c) {
  return kRow == 64 ? r * 4 + c : r * (kRow / 16) + (c ^ ((r & 1) << 2));
}
template <int kRow, bool kBf16Cache>
__device__ __forceinline__ int v_place(int r, int c) {
  if (kRow == 64) return (r >> 1) * 8 + ((((r & 1) << 2) + c) ^ (((r >> 1) & 3) << 1));
  return r * (kRow / 16) + (kBf16Cache ? c ^ (r & 7) : c ^ (((r >> 1) & 3) << 1));
}

template <int kHd, int kKind, bool kBf16, int R>
struct Shared {
  using Z = Sizes<kHd, kKind>;
  static constexpr int kQTiles = tiles_of(Parts<kKind, kBf16>::kQ, R);
  static constexpr int kQBytes = kHd / 16 * kQTiles * 512;
  static constexpr int kRingAt = kQBytes;
  static constexpr int kStatAt = kRingAt + kWarps * Z::kSlots * Z::kSlot;
  // m and l of every warp's rows, the rows' factors, sums of the search
  static constexpr int kBytes = kStatAt + kWarps * 16 * 8 + 16 * 4 + 2 * kWarps * 8 + 32;
};

template <int kHd, int kKind, bool kBf16, int R>
__global__ void __launch_bounds__(kThreads, Sizes<kHd, kKind>::kCtas)
    attn_kernel(const AttnArgs P) {
  using Z = Sizes<kHd, kKind>;
  using Sh = Shared<kHd, kKind, kBf16, R>;
  using T = typename std::conditional<kBf16, __nv_bfloat16, float>::type;
  constexpr bool kHalf = kKind != kKvBf16;
  constexpr int kTT = Z::kTT, kRow = Z::kRow, kSlots = Z::kSlots, kNJ = kTT / 8;
  constexpr int kQP = Parts<kKind, kBf16>::kQ, kPP = Parts<kKind, kBf16>::kP;
  constexpr int kQT = Sh::kQTiles, kPT = tiles_of(kPP, R);
  constexpr int kVec = 16 / Z::kBytes;  // elements of 16 bytes
  constexpr int kTiles = kHd / 8;       // column tiles of the sums
  extern __shared__ __align__(128) unsigned char smem[];

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int nrt = (P.M * P.group + 8 * R - 1) / (8 * R), items = P.c.kvh * nrt;
  uint32_t *const qs = reinterpret_cast<uint32_t *>(smem);
  float2 *const stat = reinterpret_cast<float2 *>(smem + Sh::kStatAt);  // [warp][16]
  float *const factor = reinterpret_cast<float *>(stat + kWarps * 16);  // [16]
  long long *const room = reinterpret_cast<long long *>(factor + 16);
  int *const found = reinterpret_cast<int *>(room + 2 * kWarps);  // [3]

  // ---- this CTA's share: chunks [u0, u1) of the list, from sequence b0 on
  auto chunks = [&](int b, int &start) {
    return (length_of(P, b, start) + Z::kChunk - 1) / Z::kChunk;
  };
  long long total = 0, none = 0;
  for (int b = tid; b < P.B; b += kThreads) {
    int start;
    const int n = chunks(b, start);
    total += n;
    if (P.err && blockIdx.x == 0 && n == 0 && !(P.counts && P.counts[b] == 0)) *P.err = 1;
  }
  block_sums(total, none, room);
  total *= items;
  if (total == 0) return;
  const Share share{total, (int)min((long long)gridDim.x, total)};
  if ((int)blockIdx.x >= share.ctas) return;
  const long long u0 = share.first(blockIdx.x), u1 = share.first(blockIdx.x + 1);
  long long before = 0;  // chunks (of one item each) of the sequences before
  for (int base = 0; base < P.B; base += kThreads) {
    int start, n = base + tid < P.B ? chunks(base + tid, start) : 0, up = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(kFull, up, d);
      if (lane >= d) up += x;
    }
    __syncthreads();
    if (lane == 31) room[warp] = up;
    __syncthreads();
    long long lo = before;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) lo += room[w];
      before += room[w];
    }
    lo = (lo + up - n) * items;
    if (n && u0 >= lo && u0 < lo + (long long)n * items) {
      found[0] = base + tid;
      found[1] = (int)((u0 - lo) / n);
      found[2] = (int)((u0 - lo) % n);
    }
    if (before * items > u0) break;
  }
  __syncthreads();

  // ---- a walk over the share: (sequence, item, chunk), `left` chunks to go
  struct Walk {
    int b, j, c, n, len, start;
    long long left;
  };
  auto enter = [&](Walk &w) {
    w.len = length_of(P, w.b, w.start);
    w.n = (w.len + Z::kChunk - 1) / Z::kChunk;
  };
  auto next_item = [&](Walk &w) {  // (only while chunks are left)
    w.c = 0;
    if (++w.j == items) {
      w.j = 0;
      do {
        ++w.b;
        enter(w);
      } while (w.n == 0);
    }
  };
  Walk ahead{found[0], found[1], found[2], 0, 0, 0, u1 - u0};
  enter(ahead);
  Walk here = ahead;

  // ---- the copies: this warp's tiles in order, K and V of each in turn
  const uint32_t ring =
      (uint32_t)__cvta_generic_to_shared(smem + Sh::kRingAt) + warp * (kSlots * Z::kSlot);
  constexpr int kCpr = kRow / 16;             // 16-byte units of a row
  constexpr int kIters = kTT * kCpr / 32;     // of a lane, for K or V of a tile
  constexpr int kHalves = kTT / 16;           // a tile's pages: one for 16 positions
  static_assert(kIters % kHalves == 0, "a lane's unit lies in one page");
  const int page_mask = (1 << P.c.page_shift) - 1;
  uint32_t bad = 0;            // slots with a page that is not there
  int put = 0;                 // the slot of the next unit
  bool v_next = false;         // the unit is V of the tile whose K went before
  long long row_at[kHalves];   // the tile's first rows in the cache, -1: none
  int rows_on = 0;             // positions of the tile that are there
  int pages[kHalves];          // of the next tile, asked for a tile ahead
  auto seek = [&]() {          // to the next chunk in which this warp has a tile
    while (ahead.left > 0 && (ahead.c * kWarps + warp) * kTT >= ahead.len) {
      --ahead.left;
      if (++ahead.c == ahead.n && ahead.left > 0) next_item(ahead);
    }
    if (ahead.left > 0) {
      const int pos = (ahead.c * kWarps + warp) * kTT;
#pragma unroll
      for (int i = 0; i < kHalves; ++i) {
        const int col = (pos + 16 * i) >> P.c.page_shift;
        pages[i] = pos + 16 * i < ahead.len ? __ldg(P.table + (size_t)ahead.b * P.cols + col) : 0;
      }
    }
  };
  auto issue = [&]() {
    if (ahead.left > 0 || v_next) {
      const uint32_t slot = ring + put * Z::kSlot;
      if (!v_next) {
        const int pos = (ahead.c * kWarps + warp) * kTT;
        rows_on = min(ahead.len - pos, kTT);
        bad &= ~(1u << put);
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
          const bool ok = (unsigned)pages[i] < (unsigned)P.c.pages;
          if (!ok && 16 * i < rows_on) bad |= 1u << put;
          row_at[i] = !ok ? -1
                          : (((long long)pages[i] * P.c.kvh + ahead.j / nrt) << P.c.page_shift) +
                                ((pos + 16 * i) & page_mask);
        }
        --ahead.left;
        if (++ahead.c == ahead.n && ahead.left > 0) next_item(ahead);
      }
      const unsigned char *from = static_cast<const unsigned char *>(v_next ? P.c.v : P.c.k);
#pragma unroll
      for (int i = 0; i < kIters; ++i) {
        const int half = i / (kIters / kHalves), u = 32 * i + lane, r = u / kCpr, c = u % kCpr;
        const bool on = row_at[half] >= 0 && r < rows_on;
        const int to = v_next ? v_place<kRow, kKind == kKvBf16>(r, c) : k_place<kRow>(r, c);
        cp16(slot + 16 * to,
             from + (on ? (size_t)(row_at[half] + (r & 15)) * kRow + 16 * c : (size_t)0), on);
      }
      if (kKind != kKvBf16 && !v_next && lane < 2 * kTT / 4) {  // both scales, with K
        const int which = lane / (kTT / 4), r = 4 * (lane % (kTT / 4)), half = r / 16;
        const float *s = which ? P.c.v_scale : P.c.k_scale;
        const bool on = row_at[kHalves == 1 ? 0 : half] >= 0 && r < rows_on;
        cp16(slot + Z::kUnit + 16 * lane,
             s + (on ? (size_t)(row_at[kHalves == 1 ? 0 : half] + (r & 15)) : (size_t)0), on);
      }
      if (v_next) seek();
      v_next = !v_next;
      put = put + 1 == kSlots ? 0 : put + 1;
    }
    commit();
  };
  seek();
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) issue();

  float acc[kTiles][4];
  float m[R], l[R];
  int lim[R];  // positions that the lane's rows see
  int get = 0;

  while (here.left > 0) {
    // ---- an item's part: chunks [here.c, here.c + n)
    const int c0 = here.c, n = (int)min((long long)(here.n - here.c), here.left);
    const int b = here.b, h = here.j / nrt, row0 = (here.j % nrt) * 8 * R;
    const int rows = min(8 * R, P.M * P.group - row0);
    const int len = here.len, start = here.start, seen_by_all = start + 1 + row0 / P.group;

    // q's rows as the products' operands: warp w has rows w and w + 8
    __syncthreads();  // (the last item's are read)
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = warp + 8 * i, row = row0 + r;
      const int mt = row / P.group, head = h * P.group + row - mt * P.group;
      const T *src = static_cast<const T *>(P.q) +
                     (((size_t)b * P.M + mt) * P.qh + head) * kHd;
      float x[kHd == 256 ? 2 : 1][4] = {};
      constexpr int kQuads = kHd == 256 ? 2 : 1;
#pragma unroll
      for (int e = 0; e < kQuads; ++e)
        if (r < rows && lane + 32 * e < kHd / 4) load4(src + 4 * (lane + 32 * e), x[e]);
      float f = P.scale;
      if (kHalf) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < kQuads; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(x[e][k]) & 0x7fffffffu);
        top = __reduce_max_sync(kFull, top);
        // below 2^(ex + 1), or not finite: as it is
        const int ex = top < 0x7f800000u ? max((int)(top >> 23) - 127, -126) : 0;
        const int up = 13 - ex;  // by two factors that are floats
        const float f0 = __int_as_float((up / 2 + 127) << 23);
        const float f1 = __int_as_float((up - up / 2 + 127) << 23);
#pragma unroll
        for (int e = 0; e < kQuads; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[e][k] = x[e][k] * f0 * f1;
        f = f / f0 / f1;
      }
      if (lane == 0) factor[r] = f;
#pragma unroll
      for (int e = 0; e < kQuads; ++e) {
        const int d = 4 * (lane + 32 * e);
        if (d < kHd) {
          // channels d .. d + 3: product ks, lane 4 (r % 8) + tq, both pairs
          const int ks = d / (4 * kVec) * (kVec / 4) + d % kVec / 4, tq = d / kVec % 4;
          uint32_t lo[kQP], hi[kQP];
          cut<kHalf, kQP>(x[e][0], x[e][1], lo);
          cut<kHalf, kQP>(x[e][2], x[e][3], hi);
#pragma unroll
          for (int p = 0; p < kQT * (R == 1 ? 2 : 1); ++p) {
            const int tile = R == 1 ? p / 2 : p, up = R == 1 ? p & 1 : i;
            uint32_t *to = qs + ((ks * kQT + tile) * 32 + 4 * (r & 7) + tq) * 4 + up;
            to[0] = p < kQP ? lo[p < kQP ? p : 0] : 0u;
            to[2] = p < kQP ? hi[p < kQP ? p : 0] : 0u;
          }
        }
      }
    }
    __syncthreads();
    float fac[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = kNone;
      l[i] = 0.0f;
      fac[i] = factor[g + 8 * i];
      lim[i] = start + 1 + (row0 + g + 8 * i) / P.group;
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;

    int any = 0;
    for (int c = c0; c < c0 + n; ++c) {
      const int pos = (c * kWarps + warp) * kTT;
      if (pos >= len) continue;
      any = 1;
      const bool masked = pos + kTT > seen_by_all || pos + kTT > len;
      // ---- scores of the tile
      wait_for<kSlots - 2>();
      __syncwarp();
      issue();
      uint32_t slot = ring + get * Z::kSlot;
      const bool broken = bad >> get & 1;
      float s[kNJ][4] = {};
#pragma unroll
      for (int sg = 0; sg < kHd / (4 * kVec); ++sg) {
        uint4 raw[kNJ];
#pragma unroll
        for (int j = 0; j < kNJ; ++j)
          raw[j] = lds128(slot + 16 * k_place<kRow>(8 * j + g, 4 * sg + t));
#pragma unroll
        for (int u = 0; u < kVec / 4; ++u) {
          uint32_t b0[kNJ], b1[kNJ];
#pragma unroll
          for (int j = 0; j < kNJ; ++j) {
            const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            if (kHalf) {
              widen<kKind>(w[u], b0[j], b1[j]);
            } else {
              b0[j] = w[(2 * u) & 3];
              b1[j] = w[(2 * u + 1) & 3];
            }
          }
#pragma unroll
          for (int p = 0; p < kQT; ++p) {
            const uint4 a = *reinterpret_cast<const uint4 *>(
                qs + (((sg * (kVec / 4) + u) * kQT + p) * 32 + lane) * 4);
#pragma unroll
            for (int j = 0; j < kNJ; ++j) mma<kHalf>(s[j], a, b0[j], b1[j]);
          }
        }
      }
      // ---- their maximum, weights and sums
      float x[R][kNJ][2], vs[kNJ][2], top[R];
#pragma unroll
      for (int i = 0; i < R; ++i) top[i] = kNone;
#pragma unroll
      for (int j = 0; j < kNJ; ++j) {
        float2 ks = make_float2(1.0f, 1.0f), lv = make_float2(0.0f, 0.0f);
        if (kHalf) {
          const uint2 a = lds64(slot + Z::kUnit + 4 * (8 * j + 2 * t));
          const uint2 v = lds64(slot + Z::kUnit + 4 * kTT + 4 * (8 * j + 2 * t));
          ks = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
          vs[j][0] = __uint_as_float(v.x);
          vs[j][1] = __uint_as_float(v.y);
          lv = make_float2(rough_log2(vs[j][0]) - 12.0f, rough_log2(vs[j][1]) - 12.0f);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float s0 = R == 1 ? s[j][0] + s[j][2] : s[j][2 * i];
          const float s1 = R == 1 ? s[j][1] + s[j][3] : s[j][2 * i + 1];
          x[i][j][0] = s0 * (fac[i] * ks.x);
          x[i][j][1] = s1 * (fac[i] * ks.y);
          if (masked) {
            const int at = pos + 8 * j + 2 * t;
            if (at >= lim[i] || at >= len) x[i][j][0] = -INFINITY;
            if (at + 1 >= lim[i] || at + 1 >= len) x[i][j][1] = -INFINITY;
          }
          top[i] = fmaxf(top[i], fmaxf(x[i][j][0] + lv.x, x[i][j][1] + lv.y));
        }
      }
      bool grown = false;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], 2));
        grown |= top[i] > m[i] + kSlack;
      }
      if (__any_sync(kFull, grown)) {
        float a[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float to = top[i] > m[i] + kSlack ? top[i] : m[i];
          a[i] = exp2_(m[i] - to);
          m[i] = to;
          l[i] *= a[i];
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          acc[i][0] *= a[0];
          acc[i][1] *= a[0];
          acc[i][2] *= a[R - 1];
          acc[i][3] *= a[R - 1];
        }
      }
      uint4 w[kTT / 16][kPT];
#pragma unroll
      for (int kk = 0; kk < kTT / 16; ++kk) {
        uint32_t pr[R][2][kPP];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int j = 2 * kk + q;
            float p0 = exp2_(x[i][j][0] - m[i]), p1 = exp2_(x[i][j][1] - m[i]);
            float w0 = kHalf ? p0 * vs[j][0] : p0, w1 = kHalf ? p1 * vs[j][1] : p1;
            if (masked) {  // (a masked scale or key may be anything)
              const int at = pos + 8 * j + 2 * t;
              if (at >= lim[i] || at >= len) p0 = w0 = 0.0f;
              if (at + 1 >= lim[i] || at + 1 >= len) p1 = w1 = 0.0f;
            }
            l[i] += p0 + p1;
            cut<kHalf, kPP>(w0, w1, pr[i][q]);
          }
#pragma unroll
        for (int p = 0; p < kPT; ++p) {
          if (R == 1)
            w[kk][p] = make_uint4(pr[0][0][2 * p], 2 * p + 1 < kPP ? pr[0][0][(2 * p + 1) % kPP] : 0u,
                                  pr[0][1][2 * p], 2 * p + 1 < kPP ? pr[0][1][(2 * p + 1) % kPP] : 0u);
          else
            w[kk][p] = make_uint4(pr[0][0][p], pr[R - 1][0][p], pr[0][1][p], pr[R - 1][1][p]);
        }
      }
      if (broken) {
        if (P.err) *P.err = 1;
#pragma unroll
        for (int i = 0; i < R; ++i) l[i] = __uint_as_float(0x7fc00000u);
      }
      get = get + 1 == kSlots ? 0 : get + 1;

      // ---- the sums over v
      wait_for<kSlots - 2>();
      __syncwarp();
      issue();
      slot = ring + get * Z::kSlot;
      if (kKind == kKvBf16 && masked && P.M > 1) {
        // A row that some tokens do not see must not reach them, whatever it
        // holds: one with an element that is not finite is taken out, and the
        // rows that see it become NaN by their sum.
        for (int r = 0; r < kTT; ++r) {
          if (pos + r <= start || pos + r >= len) continue;
          bool odd = false;
          for (int c4 = lane; c4 < kCpr; c4 += 32) {
            const uint4 q = lds128(slot + 16 * v_place<kRow, true>(r, c4));
            const uint32_t e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              odd |= (e[k] & 0x7f80u) == 0x7f80u || (e[k] & 0x7f800000u) == 0x7f800000u;
          }
          if (!__any_sync(kFull, odd)) continue;
          for (int c4 = lane; c4 < kCpr; c4 += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             slot + 16 * v_place<kRow, true>(r, c4)),
                         "r"(0u)
                         : "memory");
#pragma unroll
          for (int i = 0; i < R; ++i)
            if (pos + r < lim[i]) l[i] = __uint_as_float(0x7fc00000u);
        }
        __syncwarp();
      }
      if (kKind == kKvBf16) {
#pragma unroll
        for (int kk = 0; kk < kTT / 16; ++kk)
#pragma unroll
          for (int i = 0; i < kTiles / 2; ++i) {
            uint32_t v0, v1, v2, v3;
            const int r = 16 * kk + (lane & 15), cc = 2 * i + (lane >> 4);
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v0), "=r"(v1), "=r"(v2), "=r"(v3)
                         : "r"(slot + 16 * v_place<kRow, true>(r, cc)));
#pragma unroll
            for (int p = 0; p < kPT; ++p) {
              mma<false>(acc[2 * i], w[kk][p], v0, v1);
              mma<false>(acc[2 * i + 1], w[kk][p], v2, v3);
            }
          }
      } else {
        // four positions a lane, 16 channels of each (8 of 64): bytes of
        // neighbouring positions side by side make the pairs of an operand
        constexpr int kWords = kHd == 64 ? 2 : 4;
#pragma unroll
        for (int kk = 0; kk < kTT / 16; ++kk)
#pragma unroll
          for (int i = 0; i < (kHd == 256 ? 2 : 1); ++i) {
            uint32_t e[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int r = 16 * kk + 2 * t + (q & 1) + 8 * (q >> 1);
              if (kHd == 64) {
                const uint2 v = lds64(slot + 16 * v_place<kRow, false>(r, g >> 1) + 8 * (g & 1));
                e[q][0] = v.x; e[q][1] = v.y;
              } else {
                const uint4 v = lds128(slot + 16 * v_place<kRow, false>(r, g + 8 * i));
                e[q][0] = v.x; e[q][1] = v.y; e[q][2] = v.z; e[q][3] = v.w;
              }
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
              uint32_t b0[4], b1[4];
              widen<kKind>(prmt(e[0][k], e[1][k], 0x5140), b0[0], b0[1]);
              widen<kKind>(prmt(e[0][k], e[1][k], 0x7362), b0[2], b0[3]);
              widen<kKind>(prmt(e[2][k], e[3][k], 0x5140), b1[0], b1[1]);
              widen<kKind>(prmt(e[2][k], e[3][k], 0x7362), b1[2], b1[3]);
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int p = 0; p < kPT; ++p)
                  mma<true>(acc[16 * i + 4 * k + q], w[kk][p], b0[q], b1[q]);
            }
          }
      }
      get = get + 1 == kSlots ? 0 : get + 1;
    }

    // ---- the warps' sums meet.  The slot that was read last is this warp's
    // room: the copies that are under way go to the others.
    const bool whole = c0 == 0 && n == here.n;
    here.left -= n;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      l[i] += __shfl_xor_sync(kFull, l[i], 1);
      l[i] += __shfl_xor_sync(kFull, l[i], 2);
      if (t == 0) stat[warp * 16 + g + 8 * i] = make_float2(m[i], any ? l[i] : 0.0f);
    }
    const int mine = get == 0 ? kSlots - 1 : get - 1;
    float4 *const own = reinterpret_cast<float4 *>(smem + Sh::kRingAt) +
                        (warp * kSlots + mine) * (Z::kSlot / 16);
    // 16-byte unit q of a row of fp32 sums
    auto unit = [](int r, int q) { return r * (kHd / 4) + (q ^ (((q >> 3) ^ (r << 2)) & 7)); };
    __syncwarp();
    int *const slots = found + 4;  // [8] bytes: the warps' rooms, -1: nothing
    if (lane == 0) reinterpret_cast<signed char *>(slots)[warp] = any ? (signed char)mine : -1;
    float *const part =
        P.part + ((size_t)blockIdx.x * 2 + (c0 == 0 ? 1 : 0)) * (8 * R) * (kHd + 4);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (any) {
        if (kKind == kKvBf16) {
#pragma unroll
          for (int q = 0; q < kTiles; ++q) {
            const float a = R == 1 ? acc[q][0] + acc[q][2] : acc[q][2 * i];
            const float d = R == 1 ? acc[q][1] + acc[q][3] : acc[q][2 * i + 1];
            *(reinterpret_cast<float2 *>(own + unit(g, 2 * q + t / 2)) + (t & 1)) = make_float2(a, d);
          }
        } else {
          constexpr int kRun = kHd == 64 ? 8 : 16;  // channels side by side of a lane
#pragma unroll
          for (int q = 0; q < kTiles / 4; ++q) {
            const int blk = 4 * q / kRun, e = 4 * q % kRun;
            float a[4], d[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              a[k] = R == 1 ? acc[4 * q + k][0] + acc[4 * q + k][2] : acc[4 * q + k][2 * i];
              d[k] = R == 1 ? acc[4 * q + k][1] + acc[4 * q + k][3] : acc[4 * q + k][2 * i + 1];
            }
            const int at = (128 * blk + 2 * t * kRun + e) / 4;
            own[unit(g, at)] = make_float4(a[0], a[1], a[2], a[3]);
            own[unit(g, at + kRun / 4)] = make_float4(d[0], d[1], d[2], d[3]);
          }
        }
      }
      __syncthreads();
      for (int q = tid; q < 8 * (kHd / 4); q += kThreads) {
        const int r = q / (kHd / 4), cq = q % (kHd / 4), row = row0 + r + 8 * i;
        if (r + 8 * i >= rows) continue;
        float top = kNone, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w * 16 + r + 8 * i].x);
        float o[4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const int sl = reinterpret_cast<const signed char *>(slots)[w];
          if (sl < 0) continue;
          const float2 ml = stat[w * 16 + r + 8 * i];
          const float f = exp2_(ml.x - top);
          sum += ml.y * f;
          const float4 v = reinterpret_cast<const float4 *>(
              smem + Sh::kRingAt)[(w * kSlots + sl) * (Z::kSlot / 16) + unit(r, cq)];
          o[0] += v.x * f; o[1] += v.y * f; o[2] += v.z * f; o[3] += v.w * f;
        }
        if (whole) {
          const int mt = row / P.group, head = h * P.group + row - mt * P.group;
          const size_t at = ((size_t)b * P.M + mt) * P.qh + head;
          if (mt + start >= len) continue;  // a token that the sequence has not
          const float inv = 1.0f / sum;
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] *= inv;
          store4(static_cast<T *>(P.o) + at * kHd + 4 * cq, o);
          if (P.lse && cq == 0) P.lse[at] = (top + log2f(sum)) * 0.693147180559945f;
        } else {
          float *to = part + (size_t)(r + 8 * i) * (kHd + 4);
          store4(to + 4 * cq, o);
          if (cq == 0) *reinterpret_cast<float2 *>(to + kHd) = make_float2(top, sum);
        }
      }
      __syncthreads();
    }
    here.c += n;
    if (here.left > 0) next_item(here);
  }
  wait_for<0>();
}

// Rows whose item lies in several CTAs: the parts in the CTAs' order, a row for
// each block, four groups of threads (hd 256) to sixteen over the parts.
template <int kHd, int kKind, bool kBf16, int R>
__global__ void __launch_bounds__(kThreads)
    attn_join_kernel(const AttnArgs P, int grid) {
  using Z = Sizes<kHd, kKind>;
  using T = typename std::conditional<kBf16, __nv_bfloat16, float>::type;
  constexpr int kQ = kHd / 4, kGroups = kThreads / kQ;
  __shared__ long long room[2 * kWarps];
  __shared__ float4 sums[kGroups][kQ];
  __shared__ float tops[kGroups], ls[kGroups];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, rows = P.M * P.group;
  const int nrt = (rows + 8 * R - 1) / (8 * R), items = P.c.kvh * nrt;
  const int row = blockIdx.x % rows, h = blockIdx.x / rows % P.c.kvh;
  const int b = blockIdx.x / rows / P.c.kvh;
  long long total = 0, before = 0;
  for (int i = tid; i < P.B; i += kThreads) {
    int start;
    const int n = (length_of(P, i, start) + Z::kChunk - 1) / Z::kChunk;
    total += n;
    if (i < b) before += n;
  }
  block_sums(total, before, room);
  int start;
  const int len = length_of(P, b, start), n = (len + Z::kChunk - 1) / Z::kChunk;
  const int mt = row / P.group;
  if (n == 0 || start + mt >= len) return;
  const Share share{total * items, (int)min((long long)grid, total * items)};
  const long long u = before * items + (long long)n * (h * nrt + row / (8 * R));
  const int i0 = share.of(u), i1 = share.of(u + n - 1);
  if (i0 == i1) return;
  const int q = tid % kQ, group = tid / kQ;
  const float *part = P.part + (size_t)(row % (8 * R)) * (kHd + 4);
  constexpr size_t kStep = (size_t)(8 * R) * (kHd + 4);
  auto at = [&](int i) { return part + ((size_t)i * 2 + (i == i0 ? 1 : 0)) * kStep; };
  float top = kNone, sum = 0.0f, o[4] = {};
  constexpr int kU = 4;
  for (int i = i0 + group; i <= i1; i += kU * kGroups) {
    float2 ml[kU];
    float x[kU][4];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (i + k * kGroups > i1) continue;
      ml[k] = *reinterpret_cast<const float2 *>(at(i + k * kGroups) + kHd);
      load4(at(i + k * kGroups) + 4 * q, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (i + k * kGroups > i1) continue;
      const float to = fmaxf(top, ml[k].x), f = exp2_(top - to), e = exp2_(ml[k].x - to);
      top = to;
      sum = sum * f + ml[k].y * e;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] = o[d] * f + x[k][d] * e;
    }
  }
  sums[group][q] = make_float4(o[0], o[1], o[2], o[3]);
  if (q == 0) {
    tops[group] = top;
    ls[group] = sum;
  }
  __syncthreads();
  if (group) return;
  float all = kNone;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) all = fmaxf(all, tops[i]);
  float y[4] = {};
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float f = exp2_(tops[i] - all);
    const float4 v = sums[i][q];
    sum += ls[i] * f;
    y[0] += v.x * f; y[1] += v.y * f; y[2] += v.z * f; y[3] += v.w * f;
  }
  const float inv = 1.0f / sum;
#pragma unroll
  for (int d = 0; d < 4; ++d) y[d] *= inv;
  const size_t to = ((size_t)b * P.M + mt) * P.qh + h * P.group + row - mt * P.group;
  store4(static_cast<T *>(P.o) + to * kHd + 4 * q, y);
  if (P.lse && q == 0) P.lse[to] = (all + log2f(sum)) * 0.693147180559945f;
}

// CTAs of a call: at most one share each for the longest that the table holds.
template <int kHd, int kKind>
int grid_of(int B, int M, int group, int kvh, int R, long long room) {
  using Z = Sizes<kHd, kKind>;
  const long long nrt = (M * group + 8 * R - 1) / (8 * R);
  const long long most = (room + Z::kChunk - 1) / Z::kChunk * nrt * kvh * B;
  const int all = kSms * Z::kCtas;
  return (int)(most < all ? most : all);
}

template <int kHd, int kKind, bool kBf16, int R>
cudaError_t go(const AttnArgs &P, cudaStream_t stream) {
  using Z = Sizes<kHd, kKind>;
  using Sh = Shared<kHd, kKind, kBf16, R>;
  static_assert(Sh::kBytes * Z::kCtas <= 227 * 1024 - 1024 * (Z::kCtas - 1), "shared memory");
  static_assert(Z::kSlots >= 3 && 8 * kHd * 4 <= Z::kSlot, "rings");
  const int grid = grid_of<kHd, kKind>(P.B, P.M, P.group, P.c.kvh, R,
                                       (long long)P.cols << P.c.page_shift);
  const long long rows = (long long)P.B * P.M * P.qh;
  if (rows > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (grid == 0) return cudaSuccess;
  const auto kernel = attn_kernel<kHd, kKind, kBf16, R>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Sh::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, P);
  if (e != cudaSuccess || grid == 1) return e;
  cfg.gridDim = dim3((unsigned)rows);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<kHd, kKind, kBf16, R>, P, grid);
}

// Up to 8 rows of an item share a tile with their second parts.
inline int tile_rows(int M, int group) { return (long long)M * group <= 8 ? 1 : 2; }

template <int kHd, int kKind>
cudaError_t by_type(const AttnArgs &P, bool bf16, cudaStream_t stream) {
  if (tile_rows(P.M, P.group) == 1)
    return bf16 ? go<kHd, kKind, true, 1>(P, stream) : go<kHd, kKind, false, 1>(P, stream);
  return bf16 ? go<kHd, kKind, true, 2>(P, stream) : go<kHd, kKind, false, 2>(P, stream);
}

template <int kHd>
cudaError_t launch(const AttnArgs &P, bool bf16, cudaStream_t stream) {
  return P.c.kind == kKvBf16   ? by_type<kHd, kKvBf16>(P, bf16, stream)
         : P.c.kind == kKvInt8 ? by_type<kHd, kKvInt8>(P, bf16, stream)
                               : by_type<kHd, kKvE4m3>(P, bf16, stream);
}

// Bytes of the parts: two for each CTA.
template <int kHd>
size_t bytes(int kind, int M, int group) {
  const int R = tile_rows(M, group);
  const int ctas = kSms * (kind == kKvBf16 ? Sizes<kHd, kKvBf16>::kCtas : Sizes<kHd, kKvInt8>::kCtas);
  return (size_t)ctas * 2 * (8 * R) * (kHd + 4) * 4;
}

}  // namespace attn

cudaError_t launch_attn_64(const AttnArgs &P, bool bf16, cudaStream_t stream);
cudaError_t launch_attn_128(const AttnArgs &P, bool bf16, cudaStream_t stream);
cudaError_t launch_attn_256(const AttnArgs &P, bool bf16, cudaStream_t stream);

}  // namespace gdn
