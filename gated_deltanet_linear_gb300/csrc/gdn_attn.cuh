// Attention of new tokens over a paged key-value cache, for sm_103a
// (gdn_attn_step_m): the kernels, compiled for one head size by each of
// gdn_attn_64.cu, gdn_attn_128.cu and gdn_attn_256.cu.
//
// What they compute (sequence b, key head h, row r = (token m, query head of
// h's group)):
//     s_j = scale q_r . k_j,  j <= start[b] + m;
//     o_r = sum_j e^{s_j} v_j / sum_j e^{s_j}.
// One pass over the cache: each warp keeps a reference m_r (the largest score when
// it was last set), the sum l_r of the weights p_j = 2^{s_j log2 e - m_r} and the sums
// over v of its rows.  Parts of a sequence meet by
//     l = sum_p l_p 2^{m_p - m},  o = sum_p acc_p 2^{m_p - m} / l.
//
// Work split.  A sequence's positions are cut into chunks, a tile of 16 to 64
// positions for each warp; chunks of all (sequence, head, row tile) items follow one
// another and every CTA takes an equal, contiguous share of that list, found from
// the lengths on the device.  An item that lies within one CTA is finished there;
// of the others a CTA leaves at most two parts in the workspace, which a second,
// small kernel adds in order.  So the workspace does not grow with the batch,
// ragged batches fill the GPU, and the same lengths give the same bits.  (Joining
// in the CTA that comes last: its counters took 20 us where 33 CTAs met, marks
// without counters 14 us in place of 9 for one sequence, and 2 us less for 64.)
//
// Loads.  Each warp copies its own tiles, K and V in turn, 16 bytes a lane
// (cp.async) into its own ring: no barrier within an item, and the copies of the
// next item are under way while this one is joined.  About 100 KB an SM are in
// flight.  16-byte units are stored permuted, so that the reads below meet no bank
// twice.
//
// Products: mma.sync m16n8k16 with fp32 sums, positions (then channels) as the 16
// rows, 8 query rows as the columns, so that 8 rows waste nothing.  tcgen05 would
// want 8-bit codes widened in shared memory first, twice the bytes of the copies;
// here they are widened in registers.  The channels of a product may come in any
// order as long as q follows, so a lane reads 16 bytes of a K row and has 4 (bf16:
// 2) products' worth of operands.  The weights come out as the products' columns
// by a transposition of 8 x 8 tiles in registers; V is read by transposed 16-bit
// tiles, whose halves (8 bits) are two neighbouring channels.
//   8 bits   codes are exact in fp16; q of a row is scaled by a power of two to
//            below 2^14 and cut into fp16 parts (bf16: one, exact for elements
//            above 2^-28 of the row's largest; fp32: two, 22 bits); scales are
//            applied to the scores, and to the weights: w_j = p_j vscale_j 2^k_r.  k_r
//            is set with the reference so that the largest w is from 2^12 on, and
//            anew when one passes 65000: an fp16 part ends 2^-37 of the largest
//            below.  w as two parts (22 bits).  The sums over v are in units of
//            2^(m_r - k_r), l_r in those of 2^m_r: the scales of v, from 0 to any
//            size, have no say in the weights' sum (one reference for both,
//            log2 vscale above the scores, let l leave the floats over rows of zeros;
//            64 sequences of 4096, int8: 95 us with one, 97 with two).
//   bf16     q one bf16 part or (fp32) three, weights three parts (24 bits).
// The weights keep these parts for bf16 tokens too: a single fp16 part (2^-11 of
// each weight) or two bf16 ones (2^-17) put a bf16 result on the other side of a
// border many times as often as fp32 sums do (64 sequences of 4096 in int8: 91 us
// and 1.1e-3 from the rounded 64-bit result with one part, 95 us and 5e-5 with two;
// 24 rows over bf16, 53 and 58 us).
//
// Measured (uniform lengths, copies from HBM at 6.8 TB/s): bf16 caches 91 to 94 %
// of the copy rate with 4 rows a head, 8 bits 80 to 89 % (64 channels 72), where the
// widening's integer operations and the weights fill 62 % of the issue slots.  9 to
// 24 rows a head 30 to 55 % (bf16 caches 53 to 72): one CTA of 8 warps holds the sums,
// two warps a scheduler, and waits for its own products.  More rows take a pass over
// keys and values for every 24 (or 16) of them: 64 tokens x 6 heads 4 % over int8.
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
constexpr float kNone = -3e30f;  // the reference of rows that have seen nothing: below any score
constexpr int kUp = 12;           // weights times scales (8 bits) are brought to 2^12,
constexpr float kTop = 65000.0f;  // and weights and these may grow to this before they are again,
constexpr int kFar = 126;         // by factors from 2^-126 to 2^126.  Sums over v are taken
constexpr float kLarge = 0x1p80f, kSmall = 0x1p-60f;  // back by those between these: 2^31 weights of
                                                      // up to 2^16 x 448 / kSmall stay floats
constexpr int kSms = 152;

// Sizes of a variant: R tiles of 8 rows.  kS warps share a tile of positions (a
// team): each takes its share of them for the scores, and its share of the
// channels for the sums over v, so that the sums of 24 rows of 256 channels fit its
// registers (4 tokens x 24 rows of 16 sequences, fp32 tokens, when they came: 94 us by
// single warps with 16 rows, 64 by teams with 24).
template <int kHd, int kKind, int R>
struct Sizes {
  static constexpr int kBytes = kKind == kKvBf16 ? 2 : 1;
  static constexpr int kRow = kHd * kBytes;               // bytes of a row
  static constexpr int kS = R > 1 && kHd == 256 && kKind != kKvBf16 ? 2 : 1;
  // CTAs an SM: two of 128 registers a lane, or one
  static constexpr int kCtas = kHd == 64 || (R == 1 && kRow <= 256) ? 2 : 1;
  static constexpr int kTeams = kWarps / kS;
  // positions of a tile: as many as leave a ring of three parts (32 against 16 for
  // 128 channels of 8 bits: 100 us, 114; 64 against 32 for 64 channels: 107, 118; both
  // with weights of one part) and fit the registers (64 channels, 16 rows: 16)
  static constexpr int kTile = kRow == 64 && R == 1 ? 64 : kS == 2 || (kCtas == 1 && kRow <= 256)    ? 32
                               : kRow > 128 || (kHd == 64 && R == 2) ? 16
                                                                     : 32;
  static constexpr int kOwn = kTile / kS;                 // of them a warp's, for the scores
  static constexpr int kVHd = kHd / kS;                   // a warp's channels of v
  static constexpr int kVRow = kRow / kS;
  static constexpr int kUnit = kOwn * kRow;               // a warp's part of K or V
  static constexpr int kSlot = kUnit + (kKind == kKvBf16 ? 0 : 8 * kOwn);  // and scales
  // a warp's ring: three parts or more (teams: beside their q)
  static constexpr int kRing = kRow == 64 && R == 1 ? 13 * 1024 + 512 : kCtas == 2 ? 13 * 1024
                               : kS == 2  ? (R == 2 ? 21 : 17) * 1024
                                          : 25 * 1024 + 512;
  static constexpr int kSlots = kRing / kSlot;
  static constexpr int kChunk = kTeams * kTile;
  // channels of 8 rows of fp32 sums that a slot holds
  static constexpr int kStage = kSlot >= 32 * kVHd ? kVHd : kVHd / 2;
};

// Parts of q and of the weights.
template <int kKind, bool kBf16>
struct Parts {
  static constexpr int kQ = kKind == kKvBf16 ? (kBf16 ? 1 : 3) : (kBf16 ? 1 : 2);
  static constexpr int kP = kKind == kKvBf16 ? 3 : 2;
};

// A CTA's share of the chunks, and where an item's parts lie.
struct Share {
  long long total;
  int ctas;
  // (products below 2^32: a 64-bit division takes several hundred cycles)
  __device__ bool small() const { return total < (1 << 23); }
  __device__ long long first(int cta) const {
    if (ctas == total) return cta;
    return small() ? (long long)((unsigned)total * (unsigned)cta / (unsigned)ctas) : total * cta / ctas;
  }
  __device__ int of(long long unit) const {
    return small() ? (int)((((unsigned)unit + 1) * (unsigned)ctas - 1) / (unsigned)total)
                   : (int)(((unit + 1) * ctas - 1) / total);
  }
};

// An item that begins in a CTA and ends in another: what attn_join_kernel has to
// know of it (last < 0: none).
struct __align__(16) Split {
  int last;  // the last CTA with a part of it
  int b, h, row0, start, len, room[2];
};
constexpr size_t kSplitBytes = 2 * kSms * sizeof(Split);

// Positions that a sequence's new tokens see, and its first new one; 0 where
// there is nothing to do.
__device__ __forceinline__ int length_of(const AttnArgs &P, int b, int &start) {
  start = P.start[b];
  const int n = P.counts ? P.counts[b] : P.M;
  const long long room = (long long)P.cols << P.c.page_shift;
  if (n <= 0 || n > P.M || start < 0 || (long long)start + n > room) return 0;
  return start + n;
}

// Units of an item in the list: its chunks and one more without positions, which
// is what its start and its join cost (64 sequences of up to 8192: 113 us
// without, 103 with it).  A share that would start with such a unit starts behind
// it: an item whose chunks lie in one CTA is finished there.
template <class Z>
__host__ __device__ __forceinline__ int units_of(int len) {
  return (len + Z::kChunk - 1) / Z::kChunk + (len > 0);
}

__device__ __forceinline__ void cp16(uint32_t to, const void *from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp16(uint32_t to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
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

// c += a b: 16 by 8 by 16; fp16 or bf16.
template <bool kHalf>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, const uint2 &b) {
  if (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

// The two warps of a team.
__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, 64;" ::"r"(team + 1) : "memory");
}

// An 8 x 8 tile of 16-bit numbers, transposed among the lanes.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four codes as two pairs of fp16: bytes 0 and 2, 1 and 3 (e4m3: 0 and 1, 2 and 3).
template <int kKind>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &even, uint32_t &odd) {
  if (kKind == kKvInt8) {
    // u = code + 128 behind the bits of 1024, which is 1024 + u; less 1152
    even = (w & 0x00ff00ffu) ^ 0x64806480u;
    odd = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 off = __half2(__half_raw{0x6480}, __half_raw{0x6480});
    __half2 a = __hsub2(*reinterpret_cast<__half2 *>(&even), off);
    __half2 b = __hsub2(*reinterpret_cast<__half2 *>(&odd), off);
    even = *reinterpret_cast<uint32_t *>(&a);
    odd = *reinterpret_cast<uint32_t *>(&b);
  } else {
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(even), "=r"(odd)
        : "r"(w));
  }
}
// Bytes 0 and 2, 1 and 3 of any kind.
template <int kKind>
__device__ __forceinline__ void widen_v(uint32_t w, uint32_t &even, uint32_t &odd) {
  widen<kKind>(kKind == kKvInt8 ? w : prmt(w, w, 0x3120), even, odd);
}

// Two numbers as pairs of 16-bit parts: p[0] the nearest, p[i] of what is left.
// kMost: of any size; the nearest bf16 to the largest floats would be infinite (what is
// not finite stays so by its second part).
template <bool kHalf, int kN, bool kMost = false>
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
      constexpr float kTop16 = 0x1.fep127f;
      const bool most = kMost && kN > 1 && i == 0;
      const __nv_bfloat162 h =
          __floats2bfloat162_rn(most ? fminf(fmaxf(x, -kTop16), kTop16) : x,
                                most ? fminf(fmaxf(y, -kTop16), kTop16) : y);
      p[i] = *reinterpret_cast<const uint32_t *>(&h);
      if (i + 1 < kN) {
        x -= __uint_as_float(p[i] << 16);
        y -= __uint_as_float(p[i] & 0xffff0000u);
      }
    }
  }
}

// 2^n for whole n from -126 on; 0 below, 2^127 above.
__device__ __forceinline__ float power(float n) {
  return __int_as_float((int)(fminf(fmaxf(n, -127.0f), 127.0f) + 127.0f) << 23);
}
// The floor of log2 x, x >= 0; -127 for numbers below the normal ones, 128 for infinity.
__device__ __forceinline__ float whole_log2(float x) {
  return (float)((__float_as_int(x) >> 23) - 127);
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

// Where a 16-byte unit of a row lies in a tile: in its row (rows of 64 bytes of
// V: in its pair of rows), permuted by an exclusive or with bits of the row, so
// that the reads meet no bank twice.
template <int kRow>
__host__ __device__ constexpr int k_twist(int r) {
  return kRow == 64 ? 0 : (r & 1) << 2;
}
template <int kRow>
__host__ __device__ constexpr int v_twist(int r) {
  return kRow == 64 ? (r >> 1) & 3 : r & 7;
}
template <int kRow>
__device__ __forceinline__ int k_place(int r, int c) {
  return r * (kRow / 16) + (c ^ k_twist<kRow>(r));
}
template <int kRow>
__device__ __forceinline__ int v_place(int r, int c) {
  return (r * (kRow / 16) + c) ^ v_twist<kRow>(r);
}

template <int kHd, int kKind, bool kBf16, int R>
struct Shared {
  using Z = Sizes<kHd, kKind, R>;
  static constexpr int kQBytes = kHd / 16 * Parts<kKind, kBf16>::kQ * R * 256;
  static constexpr int kRingAt = kQBytes;
  static constexpr int kStatAt = kRingAt + kWarps * Z::kSlots * Z::kSlot;
  // m, l and the weights' factor of every warp's rows, the rows' factors, counts of
  // the search
  static constexpr int kWeightsAt =
      kStatAt + kWarps * 8 * R * 12 + 8 * R * 4 + 2 * kWarps * 8 + 48;
  // between the warps of a team: maxima, and a tile's weights
  static constexpr int kWeights = Z::kOwn / 16 * R * Parts<kKind, kBf16>::kP * 256;
  static constexpr int kBytes =
      kWeightsAt + (Z::kS == 1 ? 0 : kWarps * (2 * kWeights + 2 * 8 * R * 4 + 8));
};

template <int kHd, int kKind, bool kBf16, int R>
__global__ void __launch_bounds__(kThreads, Sizes<kHd, kKind, R>::kCtas)
    attn_kernel(const AttnArgs P) {
  using Z = Sizes<kHd, kKind, R>;
  using Sh = Shared<kHd, kKind, kBf16, R>;
  using T = typename std::conditional<kBf16, __nv_bfloat16, float>::type;
  constexpr bool kHalf = kKind != kKvBf16;
  constexpr int kRow = Z::kRow, kSlots = Z::kSlots, kS = Z::kS, kTile = Z::kTile;
  constexpr int kVHd = Z::kVHd, kVRow = Z::kVRow;
  constexpr int kMT = Z::kOwn / 16, kVT = kTile / 16;  // 16 positions: of scores, of V
  constexpr int kQP = Parts<kKind, kBf16>::kQ, kPP = Parts<kKind, kBf16>::kP;
  constexpr int kVec = 16 / Z::kBytes;  // elements of 16 bytes
  constexpr int kDT = kVHd / 16;        // tiles of 16 channels
  extern __shared__ __align__(128) unsigned char smem[];

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (the same for all lanes, and known to be)
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0);
  const int lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int team = warp / kS, sub = warp % kS;
  Split *const split = reinterpret_cast<Split *>(P.part) + blockIdx.x;
  if (tid == 0) split->last = -1;
  const int nrt = (P.M * P.group + 8 * R - 1) / (8 * R), items = P.c.kvh * nrt;
  uint32_t *const qs = reinterpret_cast<uint32_t *>(smem);
  float2 *const stat = reinterpret_cast<float2 *>(smem + Sh::kStatAt);  // [warp][8 R]
  float *const units = reinterpret_cast<float *>(stat + kWarps * 8 * R);  // [warp][8 R]
  float *const factor = units + kWarps * 8 * R;                           // [8 R]
  long long *const room = reinterpret_cast<long long *>(factor + 8 * R);
  int *const found = reinterpret_cast<int *>(room + 2 * kWarps);  // [5]
  uint2 *const weights = reinterpret_cast<uint2 *>(smem + Sh::kWeightsAt);
  float *const maxima = reinterpret_cast<float *>(smem + Sh::kWeightsAt + 2 * kWarps * Sh::kWeights);
  volatile int *const flags = reinterpret_cast<int *>(maxima + 2 * kWarps * 8 * R);  // [warp][2]
  signed char *const rooms = reinterpret_cast<signed char *>(found + 8);  // [kWarps]
  signed char *const wides = rooms + kWarps;                              // [kWarps]

  // the token of a row (of M; at least M: none)
  auto token_of = [&](int row) { return P.M == 1 ? (int)(row >= P.group) : row / P.group; };

  // ---- this CTA's share: chunks [u0, u1) of the list, from sequence b0 on
  int len0 = 0, start0 = 0;  // of the sequence that this lane looks at
  auto counted = [&](int b) {
    if (b >= P.B) return 0;
    len0 = length_of(P, b, start0);
    const int n = units_of<Z>(len0);
    if (P.err && blockIdx.x == 0 && n == 0 && !(P.counts && P.counts[b] == 0)) *P.err = 1;
    return n;
  };
  auto scan = [&](int n) {  // up to this lane's, within the warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(kFull, n, d);
      if (lane >= d) n += x;
    }
    return n;
  };
  // the first sequences lane by lane, the others' sum
  long long rest = 0;
  for (int b = tid + kThreads; b < P.B; b += kThreads) rest += counted(b);
  int n0 = counted(tid), up = scan(n0);
  if (P.B > kThreads) {
#pragma unroll
    for (int d = 16; d; d >>= 1) rest += __shfl_xor_sync(kFull, rest, d);
  }
  if (lane == 31) {
    room[warp] = up;
    room[kWarps + warp] = rest;
  }
  __syncthreads();
  long long lo = 0, before = 0, total = 0;  // chunks (of one item each) before
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) lo += room[w];
    before += room[w];
    total += room[kWarps + w];
  }
  total = (total + before) * items;
  if (total == 0) return;
  const Share share{total, (int)min((long long)gridDim.x, total)};
  if ((int)blockIdx.x >= share.ctas) return;
  const long long u0 = share.first(blockIdx.x), u1 = share.first(blockIdx.x + 1);
  auto find = [&](int b, int n, long long first) {
    first *= items;
    if (n && u0 >= first && u0 < first + (long long)n * items) {
      const int j = share.small() ? (int)((unsigned)(u0 - first) / (unsigned)n)
                                  : (int)((u0 - first) / n);
      found[0] = b;
      found[1] = j;
      found[2] = (int)(u0 - first - (long long)j * n);
      found[3] = len0;
      found[4] = start0;
    }
  };
  find(tid, n0, lo + up - n0);
  for (int base = kThreads; before * items <= u0; base += kThreads) {
    n0 = counted(base + tid);
    up = scan(n0);
    __syncthreads();
    if (lane == 31) room[warp] = up;
    __syncthreads();
    lo = before;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) lo += room[w];
      before += room[w];
    }
    find(base + tid, n0, lo + up - n0);
  }
  __syncthreads();

  // ---- a walk over the share: (sequence, head, row tile, chunk)
  struct Walk {
    int b, h, rt, c, n, len, start;
    long long left;
  };
  auto enter = [&](Walk &w) {
    w.len = length_of(P, w.b, w.start);
    w.n = units_of<Z>(w.len);
  };
  auto next_item = [&](Walk &w) {  // (only while chunks are left)
    w.c = 0;
    if (++w.rt < nrt) return;
    w.rt = 0;
    if (++w.h < P.c.kvh) return;
    w.h = 0;
    do {
      ++w.b;
      enter(w);
    } while (w.n == 0);
  };
  Walk ahead{found[0], nrt == 1 ? found[1] : found[1] / nrt, nrt == 1 ? 0 : found[1] % nrt, found[2], units_of<Z>(found[3]),
             found[3], found[4], u1 - u0};
  if (ahead.c == ahead.n - 1 && --ahead.left > 0) next_item(ahead);
  Walk here = ahead;

  // ---- the copies: this warp's tiles in order, K and V of each in turn
  const uint32_t ring =
      (uint32_t)__cvta_generic_to_shared(smem + Sh::kRingAt) + warp * (kSlots * Z::kSlot);
  constexpr int kCpr = kRow / 16, kVCpr = kVRow / 16;  // 16-byte units of a row
  constexpr int kSteps = Z::kUnit / 512;               // of a warp, for its part of K or V
  const uint32_t k_lane = 16 * k_place<kRow>(lane / kCpr, lane % kCpr);
  const uint32_t v_lane = 16 * v_place<kVRow>(lane / kVCpr, lane % kVCpr);
  const int v_from = lane / kVCpr * kRow + sub * kVRow + lane % kVCpr * 16;
  const int page_mask = (1 << P.c.page_shift) - 1;
  uint32_t bad = 0;            // slots with a page that is not there
  int put = 0;                 // the slot of the next unit
  bool begun = false;          // K of a tile is under way, its V comes next
  bool full = false;           // all of the tile's positions and pages are there
  long long row_at[kVT];       // the tile's first rows in the cache, -1: none
  int rows_on = 0;             // positions of the tile that are there
  int pages[kVT];              // of the next tile, asked for a tile ahead
  auto seek = [&]() {          // to the next chunk in which this team has a tile
    while (ahead.left > 0 && (ahead.c * Z::kTeams + team) * kTile >= ahead.len) {
      --ahead.left;
      if (++ahead.c == ahead.n && ahead.left > 0) next_item(ahead);
    }
    if (ahead.left > 0) {
      const int pos = (ahead.c * Z::kTeams + team) * kTile;
#pragma unroll
      for (int i = 0; i < kVT; ++i) {
        const int col = (pos + 16 * i) >> P.c.page_shift;
        pages[i] = pos + 16 * i < ahead.len ? __ldg(P.table + (size_t)ahead.b * P.cols + col) : 0;
      }
    }
  };
  auto issue = [&](auto which_unit) {  // K of the next tile, or V of it
    constexpr bool v_next = decltype(which_unit)::value;
    if (v_next ? begun : ahead.left > 0) {
      const uint32_t slot = ring + put * Z::kSlot;
      if (!v_next) {
        const int pos = (ahead.c * Z::kTeams + team) * kTile;
        rows_on = min(ahead.len - pos, kTile);
        full = rows_on == kTile;
        bad &= ~(1u << put);
#pragma unroll
        for (int i = 0; i < kVT; ++i) {
          const bool ok = (unsigned)pages[i] < (unsigned)P.c.pages;
          if (!ok && 16 * i < rows_on) bad |= 1u << put;
          full &= ok;
          row_at[i] = !ok ? -1
                          : (((long long)pages[i] * P.c.kvh + ahead.h) << P.c.page_shift) +
                                ((pos + 16 * i) & page_mask);
        }
        --ahead.left;
        if (++ahead.c == ahead.n && ahead.left > 0) next_item(ahead);
      }
      const unsigned char *from = static_cast<const unsigned char *>(v_next ? P.c.v : P.c.k);
      // runs of 16 positions lie in one page
      constexpr int kRuns = v_next ? kVT : kMT, kPer = kSteps / kRuns;
      constexpr int kRowsStep = 32 / (v_next ? kVCpr : kCpr);
      static_assert(kSteps % kRuns == 0 && kPer >= 1, "a step's rows lie in one page");
#pragma unroll
      for (int run = 0; run < kRuns; ++run) {
        const int i = v_next ? run : kS == 1 ? run : sub;  // (kMT == 1 in teams)
        const long long at = row_at[kVT == 1 ? 0 : kS == 1 || v_next ? run : 0];
        const long long mine = kS == 1 || v_next ? at : sub ? row_at[kVT - 1] : row_at[0];
        const unsigned char *src =
            from + (size_t)max(mine, 0ll) * kRow + (v_next ? v_from : 16 * lane);
        // (a step's rows and the lane's row within it have no bit in common, so
        // their twists add up to the row's)
        auto place = [&](int j) {
          const int step = run * kPer + j, r = step * kRowsStep;
          return slot + 512 * step +
                 (v_next ? v_lane ^ (16 * v_twist<kVRow>(r))
                         : k_lane ^ (16 * k_twist<kRow>(r)));
        };
        if (full) {
#pragma unroll
          for (int j = 0; j < kPer; ++j) cp16(place(j), src + j * kRowsStep * kRow);
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int r = 16 * i + j * kRowsStep + lane / (v_next ? kVCpr : kCpr);
            const bool on = mine >= 0 && r < rows_on;
            cp16(place(j), on ? src + j * kRowsStep * kRow : from, on);
          }
        }
      }
      if (kKind != kKvBf16 && !v_next && lane < 2 * Z::kOwn / 4) {  // both scales, with K
        const int which = lane / (Z::kOwn / 4), r = 4 * (lane % (Z::kOwn / 4)) + sub * Z::kOwn;
        const float *s = which ? P.c.v_scale : P.c.k_scale;
        long long at = row_at[0];
#pragma unroll
        for (int i = 1; i < kVT; ++i) at = r >= 16 * i ? row_at[i] : at;
        const bool on = at >= 0 && r < rows_on;
        cp16(slot + Z::kUnit + 16 * lane, s + (on ? (size_t)(at + (r & 15)) : (size_t)0), on);
      }
      if (v_next) seek();
      begun = !v_next;
      put = put + 1 == kSlots ? 0 : put + 1;
    }
    commit();
  };
  // q's rows of an item, a row a warp (R times), asked for ahead of their use
  constexpr int kQuads = kHd == 256 ? 2 : 1;
  float xq[R][kQuads][4];
  auto ask_q = [&](const Walk &w) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = w.rt * 8 * R + warp + 8 * i;
      const int mt = token_of(row), head = w.h * P.group + row - mt * P.group;
      const T *src = static_cast<const T *>(P.q) + (((size_t)w.b * P.M + mt) * P.qh + head) * kHd;
#pragma unroll
      for (int e = 0; e < kQuads; ++e) {
        xq[i][e][0] = xq[i][e][1] = xq[i][e][2] = xq[i][e][3] = 0.0f;
        // (tokens that the sequence has: the others' rows may hold anything, and one
        // row's weights can have the references of all set anew)
        if (mt < w.len - w.start && lane + 32 * e < kHd / 4) load4(src + 4 * (lane + 32 * e), xq[i][e]);
      }
    }
  };
  if (here.left > 0) ask_q(here);

  constexpr std::false_type kK{};
  constexpr std::true_type kV{};
  seek();
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) {
    if (i & 1)
      issue(kV);
    else
      issue(kK);
  }

  float acc[kDT][R][4];
  float m[R][2], l[R][2];
  float gain[R][2];  // (8 bits) the power of two that weights times scales are brought up by
  int get = 0, turn = 0;  // (turn: of two buffers between the warps of a team)

  while (here.left > 0) {
    // ---- an item's part: chunks [here.c, here.c + n)
    const int c0 = here.c, n = (int)min((long long)(here.n - here.c), here.left);
    const int b = here.b, h = here.h, row0 = here.rt * 8 * R;
    const int rows = min(8 * R, P.M * P.group - row0);
    const int len = here.len, start = here.start, seen_by_all = start + 1 + row0 / P.group;

    // q's rows as the products' operands, a row a warp
    __syncthreads();  // (the last item's are read)
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = warp + 8 * i;
      float (&x)[kQuads][4] = xq[i];
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
        const int by = 13 - ex;  // in two factors that are floats
        const float f0 = __int_as_float((by / 2 + 127) << 23);
        const float f1 = __int_as_float((by - by / 2 + 127) << 23);
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
          uint32_t a[kQP], c[kQP];
          // (int8 codes come out as bytes 0 and 2, 1 and 3)
          constexpr int k1 = kKind == kKvInt8 ? 2 : 1, k2 = 3 - k1;
          cut<kHalf, kQP, true>(x[e][0], x[e][k1], a);
          cut<kHalf, kQP, true>(x[e][k2], x[e][3], c);
#pragma unroll
          for (int p = 0; p < kQP; ++p)
            reinterpret_cast<uint2 *>(qs)[((ks * kQP + p) * R + i) * 32 + 4 * (r & 7) + tq] =
                make_uint2(a[p], c[p]);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[i][e] = kNone;
        l[i][e] = 0.0f;
        gain[i][e] = 1.0f;
      }
    // positions that row r of the item sees
    auto limit = [&](int r) { return min(len, start + 1 + (row0 + r) / P.group); };
#pragma unroll
    for (int d = 0; d < kDT; ++d)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[d][i][k] = 0.0f;

    int any = 0;
    for (int c = c0; c < c0 + n; ++c) {
      const int pos = (c * Z::kTeams + team) * kTile, mypos = pos + sub * Z::kOwn;
      if (pos >= len) continue;
      const bool first = !any;
      any = 1;
      const bool masked = pos + kTile > seen_by_all || pos + kTile > len;
      // ---- scores of the tile: 16 positions by 8 rows a product
      wait_for<kSlots - 2>();
      __syncwarp();
      issue(std::bool_constant<(kSlots - 1) % 2 == 1>{});
      uint32_t slot = ring + get * Z::kSlot;
      const bool broken = bad >> get & 1;
      // (several sums where there are few, as a product waits for the last one of
      // its sum; and one for each of three parts, small parts apart from large)
      constexpr int kC = kQP == 3 ? 3 : kMT * R <= 2 ? 2 : 1;
      float part[kC][kMT][R][4] = {};
#pragma unroll
      for (int sg = 0; sg < kHd / (4 * kVec); ++sg) {
        uint4 raw[kMT][2];
#pragma unroll
        for (int j = 0; j < kMT; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            raw[j][q] = lds128(slot + 16 * k_place<kRow>(16 * j + 8 * q + g, 4 * sg + t));
#pragma unroll
        for (int u = 0; u < kVec / 4; ++u) {
          uint32_t a[kMT][4];
#pragma unroll
          for (int j = 0; j < kMT; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t w[4] = {raw[j][q].x, raw[j][q].y, raw[j][q].z, raw[j][q].w};
              if (kHalf) {
                widen<kKind>(w[u], a[j][q], a[j][2 + q]);
              } else {
                a[j][q] = w[(2 * u) & 3];
                a[j][2 + q] = w[(2 * u + 1) & 3];
              }
            }
#pragma unroll
          for (int p = 0; p < kQP; ++p)
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const uint2 bq = reinterpret_cast<const uint2 *>(
                  qs)[(((sg * (kVec / 4) + u) * kQP + p) * R + i) * 32 + lane];
#pragma unroll
              for (int j = 0; j < kMT; ++j)
                mma<kHalf>(part[(kQP > 1 ? p : u) % kC][j][i], a[j][0], a[j][1], a[j][2], a[j][3], bq);
            }
        }
      }
      // ---- their maximum, weights and sums: a lane has positions g and g + 8
      // of 16, rows 2 t and 2 t + 1 of 8
      float (&s)[kMT][R][4] = part[0];
#pragma unroll
      for (int c = kC - 1; c > 0; --c)
#pragma unroll
        for (int j = 0; j < kMT; ++j)
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) part[c - 1][j][i][k] += part[c][j][i][k];
      float ks[kMT][2], vs[kMT][2];
#pragma unroll
      for (int j = 0; j < kMT; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          ks[j][q] = vs[j][q] = 1.0f;
          if (kHalf) {
            const float *sc = reinterpret_cast<const float *>(
                smem + Sh::kRingAt + (warp * kSlots + get) * Z::kSlot + Z::kUnit);
            const int at = 16 * j + 8 * q + g;
            ks[j][q] = sc[at];
            vs[j][q] = sc[Z::kOwn + at];
          }
        }
      float f[R][2];  // a row's factor
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) f[i][e] = factor[8 * i + 2 * t + e];
      // In base 2, rounded once: the largest less the reference made of it is 0 at
      // any size.
#pragma unroll
      for (int j = 0; j < kMT; ++j)
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[j][i][k] = __fmul_rn(s[j][i][k], f[i][k & 1] * ks[j][k >> 1]);
      if (masked) {
        // Out of a row's sight: no weight, whatever key and scales may be.  A
        // value's scale that is not finite makes the rows that see it NaN by
        // their sum, and counts as 0.
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int lim = limit(8 * i + 2 * t + e) - mypos - g;
#pragma unroll
            for (int j = 0; j < kMT; ++j)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const bool seen = 16 * j + 8 * q < lim;
                if (!seen) s[j][i][2 * q + e] = -INFINITY;
                if (kHalf && seen && !(fabsf(vs[j][q]) <= 3.4e38f)) l[i][e] = __uint_as_float(0x7fc00000u);
              }
          }
#pragma unroll
        for (int j = 0; j < kMT; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (kHalf && !(fabsf(vs[j][q]) <= 3.4e38f)) vs[j][q] = 0.0f;
      }
      // Weights with the reference and the factor as they are; where one is too
      // large for that, and for the first tile, these are set anew.
      uint2 w[kVT][R][kPP];  // of the whole tile: the team's own first
      float sum[R][2];
      auto weigh = [&]() {  // true: one does not fit
        float big = 0.0f;  // (a row's sum stands for its weights; NaN are no reason)
#pragma unroll
        for (int i = 0; i < R; ++i) sum[i][0] = sum[i][1] = 0.0f;
#pragma unroll
        for (int j = 0; j < kMT; ++j)
#pragma unroll
          for (int i = 0; i < R; ++i) {
            uint32_t pr[2][kPP];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = exp2_(s[j][i][2 * q + e] - m[i][e]);
                sum[i][e] += x;
                y[e] = kHalf ? x * vs[j][q] * gain[i][e] : x;
              }
              if (kHalf) big = fmaxf(big, fmaxf(fabsf(y[0]), fabsf(y[1])));
              cut<kHalf, kPP>(y[0], y[1], pr[q]);
            }
#pragma unroll
            for (int k = 0; k < kPP; ++k)
              w[j][i][k] = make_uint2(transposed(pr[0][k]), transposed(pr[1][k]));
          }
#pragma unroll
        for (int i = 0; i < R; ++i) big = fmaxf(big, fmaxf(sum[i][0], sum[i][1]));
        return __any_sync(kFull, big > kTop) != 0;
      };
      // to the other warp of the team, with whether the weights fit
      auto hand_over = [&](bool off) {
        uint2 *const mine = weights + (warp * 2 + turn) * (Sh::kWeights / 8) + lane;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < kPP; ++k) mine[(i * kPP + k) * 32] = w[0][i][k];
        if (lane == 0) flags[warp * 2 + turn] = off;
        team_sync(team);
        return flags[(warp ^ 1) * 2 + turn] != 0;
      };
      bool off = true;
      if (!first) {
        off = weigh();
        if (kS > 1) off |= hand_over(off);
      }
      if (off) {
        // the largest of a row, over the lanes that have its positions
        auto largest = [&](float (&x)[R][2], float *shared) {
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x[i][e] = fmaxf(x[i][e], __shfl_xor_sync(kFull, x[i][e], 4));
              x[i][e] = fmaxf(x[i][e], __shfl_xor_sync(kFull, x[i][e], 8));
              x[i][e] = fmaxf(x[i][e], __shfl_xor_sync(kFull, x[i][e], 16));
              if (kS > 1 && g == 0) shared[warp * 8 * R + 8 * i + 2 * t + e] = x[i][e];
            }
          if (kS == 1) return;
          team_sync(team);
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              x[i][e] = fmaxf(x[i][e], shared[(warp ^ 1) * 8 * R + 8 * i + 2 * t + e]);
        };
        float top[R][2], a[R][2], more[R][2];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[i][e] = kNone;
#pragma unroll
            for (int j = 0; j < kMT; ++j)
#pragma unroll
              for (int q = 0; q < 2; ++q)
                top[i][e] = fmaxf(top[i][e], s[j][i][2 * q + e]);
          }
        largest(top, maxima);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float to = fmaxf(top[i][e], m[i][e]);
            more[i][e] = to - m[i][e];
            a[i][e] = exp2_(m[i][e] - to);
            m[i][e] = to;
            l[i][e] *= a[i][e];
            top[i][e] = 0.0f;
          }
        if (kHalf) {
          // The weights' unit is that of the largest weight times scale so far: it
          // does not come down, so the factor grows by no more than the
          // reference has (the sums over v are in that unit, l is in the
          // reference's: a row of zeros, whose scale is 0, moves the one alone).
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < kMT; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                  top[i][e] = fmaxf(top[i][e], exp2_(s[j][i][2 * q + e] - m[i][e]) * fabsf(vs[j][q]));
          largest(top, maxima + kWarps * 8 * R);
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float was = whole_log2(gain[i][e]);
              float to = fminf((float)kUp - whole_log2(top[i][e]), floorf(was + more[i][e]));
              to = fminf(fmaxf(to, -(float)kFar), (float)kFar);
              gain[i][e] = power(to);
              a[i][e] *= power(to - was);
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int d = 0; d < kDT; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[d][i][k] *= a[i][k & 1];
        weigh();
        if (kS > 1) {
          turn ^= 1;  // (the other has read the first ones' flag by the second barrier)
          hand_over(false);
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) l[i][e] += sum[i][e];
      if (kS > 1) {
        const uint2 *const theirs = weights + ((warp ^ 1) * 2 + turn) * (Sh::kWeights / 8) + lane;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < kPP; ++k) w[kVT - 1][i][k] = theirs[(i * kPP + k) * 32];
        turn ^= 1;
      }
      if (broken) {
        if (P.err) *P.err = 1;
#pragma unroll
        for (int i = 0; i < R; ++i) l[i][0] = l[i][1] = __uint_as_float(0x7fc00000u);
      }
      get = get + 1 == kSlots ? 0 : get + 1;

      // ---- the sums over v: 16 channels by 8 rows a product
      wait_for<kSlots - 2>();
      __syncwarp();
      issue(std::bool_constant<(kSlots - 1) % 2 == 0>{});
      slot = ring + get * Z::kSlot;
      if (kKind == kKvBf16 && masked && P.M > 1) {
        // A row that some tokens do not see must not reach them, whatever it
        // holds: one with an element that is not finite is taken out, and the
        // rows that see it become NaN by their sum.
        for (int r = 0; r < kTile; ++r) {
          if (pos + r <= start || pos + r >= len) continue;
          bool odd = false;
          for (int c4 = lane; c4 < kVCpr; c4 += 32) {
            const uint4 q = lds128(slot + 16 * v_place<kVRow>(r, c4));
            const uint32_t e[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              odd |= (e[k] & 0x7f80u) == 0x7f80u || (e[k] & 0x7f800000u) == 0x7f800000u;
          }
          if (!__any_sync(kFull, odd)) continue;
          for (int c4 = lane; c4 < kVCpr; c4 += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             slot + 16 * v_place<kVRow>(r, c4)),
                         "r"(0u)
                         : "memory");
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (pos + r < limit(8 * i + 2 * t + e)) l[i][e] = __uint_as_float(0x7fc00000u);
        }
        __syncwarp();
      }
      // Four 8 x 8 tiles of 16 bits, transposed: neighbouring positions of a
      // channel side by side (bf16), or of two channels (8 bits: two tiles of
      // 16 channels, even ones in the upper half of a product's rows).
      constexpr int kStep = kKind == kKvBf16 ? 1 : 2;
      auto products = [&](int j, int d, float (*to)[R][4]) {
        // (in teams: the own 16 positions, then the other warp's)
        const int row = kS == 1 ? 16 * j : 16 * (j ^ sub);
        uint32_t x[4];
        const int r = row + (lane & 7) + 8 * (kStep == 1 ? lane >> 4 : lane >> 3 & 1);
        const int cc = kStep == 1 ? 2 * d + (lane >> 3 & 1) : d + (lane >> 4);
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(slot + 16 * v_place<kVRow>(r, cc)));
#pragma unroll
        for (int q = 0; q < kStep; ++q) {
          uint32_t a[4] = {x[0], x[1], x[2], x[3]};
          if (kHalf) {
            widen_v<kKind>(x[2 * q], a[0], a[1]);
            widen_v<kKind>(x[2 * q + 1], a[2], a[3]);
          }
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int p = kPP - 1; p >= 0; --p)  // (small parts first)
              mma<kHalf>(to[q][i], a[0], a[1], a[2], a[3], w[j][i][p]);
        }
      };
      // A product's sum is cut off, not rounded: over long sequences that adds up,
      // so fp32 tokens make a tile's sums from 0 and add them to the others rounded
      // (24 rows of 60000 positions, 234 tiles a warp: 7e-6 to 10e-6 of o without,
      // 0.9e-6 to 1.5e-6 with, the plain fp32 form 3e-6 to 5e-6; 4 tokens x 6 heads e4m3
      // 92 and 101 us, 128 channels int8 61 and 69).  bf16 tokens do not: 1e-5 of o
      // is a 200th of its rounding (o 23e-5 from the rounded 64-bit result, the plain
      // form 19e-5, tile by tile 5e-5; 128 channels int8 59 us, tile by tile 65).
      if (kBf16) {
#pragma unroll
        for (int j = 0; j < kVT; ++j)
#pragma unroll
          for (int d = 0; d < kDT; d += kStep) products(j, d, acc + d);
      } else {
#pragma unroll
        for (int d = 0; d < kDT; d += kStep) {
          float tile[kStep][R][4] = {};
#pragma unroll
          for (int j = 0; j < kVT; ++j) products(j, d, tile);
#pragma unroll
          for (int q = 0; q < kStep; ++q)
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[d + q][i][k] += tile[q][i][k];
        }
      }
      get = get + 1 == kSlots ? 0 : get + 1;
    }

    // ---- the warps' sums meet.  The slot that was read last is this warp's
    // room: the copies that are under way go to the others.
    const bool whole = c0 == 0 && n >= here.n - 1;
    if (c0 == 0 && !whole && tid == 0) {
      const long long unit0 = u1 - here.left;  // the item's first of the list
      *split = Split{share.of(unit0 + here.n - 2), b, h, row0, start, len, {0, 0}};
    }
    here.left -= n;
    here.c += n;
    if (here.left > 0) {
      next_item(here);
      ask_q(here);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float &x = l[i][e];
        x += __shfl_xor_sync(kFull, x, 4);
        x += __shfl_xor_sync(kFull, x, 8);
        x += __shfl_xor_sync(kFull, x, 16);
        if (g == 0) {
          const int r = warp * 8 * R + 8 * i + 2 * t + e;
          stat[r] = make_float2(m[i][e], x);
          if (kHalf) units[r] = -whole_log2(gain[i][e]);
        }
      }
    if (kHalf) {
      // the sums over v as they are, but where they might leave the floats
      bool wide = false;
#pragma unroll
      for (int i = 0; i < R; ++i)
        wide |= fmaxf(gain[i][0], gain[i][1]) > kLarge || fminf(gain[i][0], gain[i][1]) < kSmall;
      wide = __any_sync(kFull, wide) != 0;
      if (lane == 0) wides[warp] = wide;
      if (!wide) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) gain[i][e] = power(-whole_log2(gain[i][e]));
#pragma unroll
        for (int d = 0; d < kDT; ++d)
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[d][i][k] *= gain[i][k & 1];
      }
    }
    const int mine = get == 0 ? kSlots - 1 : get - 1;
    if (lane == 0) rooms[warp] = any ? (signed char)mine : (signed char)-1;
    float *const own = reinterpret_cast<float *>(smem + Sh::kRingAt + (warp * kSlots + mine) * Z::kSlot);
    // 16-byte unit q of a row of fp32 sums
    constexpr int kStage = Z::kStage, kRounds = kVHd / kStage;
    auto unit = [](int r, int q) { return r * (kStage / 4) + (q ^ (((q >> 2) ^ (q >> 5) ^ r) & 7)); };
    __syncwarp();
    float *const parts =
        P.part + kSplitBytes / 4 + ((size_t)blockIdx.x * 2 + (c0 == 0 ? 1 : 0)) * (8 * R) * (kHd + 4);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int rd = 0; rd < kRounds; ++rd) {
        if (any) {
#pragma unroll
          for (int d = 0; d < kStage / 16; ++d) {
            const float (&x)[4] = acc[rd * (kStage / 16) + d][i];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (kKind == kKvBf16) {  // channels g and g + 8 of 16
                own[4 * unit(2 * t + e, 4 * d + g / 4) + (g & 3)] = x[e];
                own[4 * unit(2 * t + e, 4 * d + 2 + g / 4) + (g & 3)] = x[2 + e];
              } else {  // 2 g and 2 g + 1
                *reinterpret_cast<float2 *>(own + 4 * unit(2 * t + e, 4 * d + g / 2) + 2 * (g & 1)) =
                    make_float2(x[e], x[2 + e]);
              }
            }
          }
        }
        __syncthreads();
        for (int q = tid; q < 8 * kS * (kStage / 4); q += kThreads) {
          const int r8 = q / (kS * (kStage / 4)), cs = q / (kStage / 4) % kS, cq = q % (kStage / 4);
          const int r = r8 + 8 * i, row = row0 + r;
          if (r >= rows) continue;
          float2 ml[kWarps];
          float top = kNone, sum = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            ml[w] = stat[w * 8 * R + r];
            top = fmaxf(top, ml[w].x);
          }
          float all_in = 0.0f;  // the sums over v are in units of 2^this
          float by[kWarps];
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            by[w] = exp2_(ml[w].x - top);
            sum += ml[w].y * by[w];
          }
          if (kHalf && *reinterpret_cast<const volatile long long *>(wides) != 0) {
            all_in = -1e30f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
              all_in = fmaxf(all_in, floorf(ml[w].x - top) + (wides[w] ? units[w * 8 * R + r] : 0.0f));
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
              by[w] *= power((wides[w] ? units[w * 8 * R + r] : 0.0f) - all_in);
          }
          float o[4] = {};
#pragma unroll
          for (int w = 0; w < kWarps; w += kS) {
            const int sl = rooms[w + cs];  // (the warp that has these channels)
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (sl >= 0)
              v = reinterpret_cast<const float4 *>(
                  smem + Sh::kRingAt + ((w + cs) * kSlots + sl) * Z::kSlot)[unit(r8, cq)];
            const float f = by[w];  // (the same for a team)
            o[0] += v.x * f; o[1] += v.y * f; o[2] += v.z * f; o[3] += v.w * f;
          }
          const int ch = cs * kVHd + rd * kStage + 4 * cq;
          if (whole) {
            const int mt = token_of(row), head = h * P.group + row - mt * P.group;
            const size_t at = ((size_t)b * P.M + mt) * P.qh + head;
            if (mt + start >= len) continue;  // a token that the sequence has not
            const float inv = 1.0f / sum;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] *= inv;
            if (kHalf && all_in != 0.0f) {
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] *= power(all_in);
            }
            store4(static_cast<T *>(P.o) + at * kHd + ch, o);
            if (P.lse && ch == 0) P.lse[at] = (top + log2f(sum)) * 0.693147180559945f;
          } else {
            float *to = parts + (size_t)r * (kHd + 4);
            store4(to + ch, o);
            if (ch == 0) *reinterpret_cast<float4 *>(to + kHd) = make_float4(top, sum, all_in, 0.0f);
          }
        }
        __syncthreads();
      }
  }
  wait_for<0>();
}

// Channels 4 q on of row r of an item with parts in the CTAs i0 .. last: every
// `step`-th part from CTA i on, added in order.  The sums over v are in units of
// 2^unit, 0 but for scales far from 1.
struct Sums {
  float top = kNone, sum = 0.0f, unit = 0.0f, o[4] = {};
  __device__ __forceinline__ void rescale(float to) {
    const float f = exp2_(top - to);
    top = to;
    sum *= f;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] *= f;
  }
  __device__ __forceinline__ void add(float s, const float (&x)[4], float e) {
    sum += s * e;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] += x[d] * e;
  }
  // one more, where the units may differ
  __device__ __forceinline__ void join(float t, float s, float un, const float (&x)[4]) {
    const float to = fmaxf(top, t), f = exp2_(top - to), e = exp2_(t - to);
    const float in = fmaxf(floorf(top - to) + unit, floorf(t - to) + un);
    const float fo = f * power(unit - in), eo = e * power(un - in);
    top = to;
    unit = in;
    sum = sum * f + s * e;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = o[d] * fo + x[d] * eo;
  }
};
template <int kHd, int R, int kU, bool kHalf>
__device__ __forceinline__ Sums add_parts(const AttnArgs &P, int i0, int last, int r, int q, int i,
                                          int step) {
  constexpr size_t kPart = (size_t)(8 * R) * (kHd + 4);
  const float *part = P.part + kSplitBytes / 4 + (size_t)r * (kHd + 4);
  Sums s;
  bool units = false;
#pragma unroll 1
  for (int c = i; c <= last; c += kU * step) {
    float2 ml[kU];
    float x[kU][4], to = s.top;
#pragma unroll
    for (int k = 0; k < kU; ++k) {  // (past the end: the first one, without weight)
      const int cta = c + k * step <= last ? c + k * step : c;
      const float *from = part + ((size_t)cta * 2 + (cta == i0 ? 1 : 0)) * kPart;
      ml[k] = *reinterpret_cast<const float2 *>(from + kHd);
      if (kHalf) units |= from[kHd + 2] != 0.0f;
      load4(from + 4 * q, x[k]);
      to = fmaxf(to, ml[k].x);
    }
    s.rescale(to);
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (c + k * step <= last) s.add(ml[k].y, x[k], exp2_(ml[k].x - to));
  }
  if (kHalf && units) {  // once more, one by one
    s = Sums{};
#pragma unroll 1
    for (int c = i; c <= last; c += step) {
      const float *from = part + ((size_t)c * 2 + (c == i0 ? 1 : 0)) * kPart;
      float x[4];
      load4(from + 4 * q, x);
      s.join(from[kHd], from[kHd + 1], from[kHd + 2], x);
    }
  }
  return s;
}

template <int kHd, bool kBf16, bool kHalf>
__device__ __forceinline__ void put_row(const AttnArgs &P, Sums &s, int b, int mt, int head,
                                        int q) {
  using T = typename std::conditional<kBf16, __nv_bfloat16, float>::type;
  const float inv = 1.0f / s.sum;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    s.o[d] *= inv;
    if (kHalf && s.unit != 0.0f) s.o[d] *= power(s.unit);
  }
  const size_t to = ((size_t)b * P.M + mt) * P.qh + head;
  store4(static_cast<T *>(P.o) + to * kHd + 4 * q, s.o);
  if (P.lse && q == 0) P.lse[to] = (s.top + log2f(s.sum)) * 0.693147180559945f;
}

// Many items in several CTAs, of few parts each: kHd / 4 threads for a row of the
// one that begins in CTA blockIdx.x, if one does, as that CTA left word of it.
template <int kHd, bool kHalf, bool kBf16, int R>
__global__ void __launch_bounds__(kThreads)
    attn_join_kernel(const AttnArgs P) {
  constexpr int kQ = kHd / 4;
  // (every block waits, also one that has nothing to do: the kernel behind this
  // one waits for this one alone)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Split s = reinterpret_cast<const Split *>(P.part)[blockIdx.x];
  if (s.last < 0) return;
  const int r = blockIdx.y * (kThreads / kQ) + threadIdx.x / kQ, q = threadIdx.x % kQ;
  const int row = s.row0 + r, mt = row / P.group;
  if (r >= 8 * R || mt >= P.M || s.start + mt >= s.len) return;  // (no token of the sequence)
  Sums x = add_parts<kHd, R, 4, kHalf>(P, blockIdx.x, s.last, r, q, blockIdx.x, 1);
  put_row<kHd, kBf16, kHalf>(P, x, s.b, mt, s.h * P.group + row - mt * P.group, q);
}

// Few items of many parts (at most 32 sequences): a block for each row, which finds
// the item's CTAs from the lengths while attn_kernel runs.
template <int kHd, int kKind, bool kBf16, int R>
__global__ void __launch_bounds__(512, 2)  // (beside a CTA of attn_kernel)
    attn_join_few_kernel(const AttnArgs P, int grid) {
  using Z = Sizes<kHd, kKind, R>;
  // (what came before attn_kernel has ended, and attn_kernel writes no lengths)
  const int rows = P.M * P.group, lane = threadIdx.x & 31;
  const int nrt = (rows + 8 * R - 1) / (8 * R), items = P.c.kvh * nrt;
  const int row = blockIdx.x % rows, h = blockIdx.x / rows % P.c.kvh;
  const int b = blockIdx.x / rows / P.c.kvh, mt = row / P.group;
  int start = 0, len = lane < P.B ? length_of(P, lane, start) : 0, up = units_of<Z>(len);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(kFull, up, d);
    if (lane >= d) up += x;
  }
  const long long total = (long long)__shfl_sync(kFull, up, 31) * items;
  start = __shfl_sync(kFull, start, b);
  len = __shfl_sync(kFull, len, b);
  const int n = units_of<Z>(len);
  const long long before = __shfl_sync(kFull, up, b) - n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (n == 0 || start + mt >= len) return;
  const Share share{total, (int)min((long long)grid, total)};
  const long long u = before * items + (long long)n * (h * nrt + row / (8 * R));
  const int i0 = share.of(u), last = share.of(u + n - 2);
  if (i0 == last) return;
  // streams of parts, joined in their order
  constexpr int kQ = kHd / 4, kGroups = 512 / kQ;
  constexpr bool kHalf = kKind != kKvBf16;
  __shared__ Sums sums[kGroups][kQ];
  const int q = threadIdx.x % kQ, group = threadIdx.x / kQ;
  const Sums mine = add_parts<kHd, R, 8, kHalf>(P, i0, last, row % (8 * R), q, i0 + group, kGroups);
  sums[group][q] = mine;
  const bool units = __syncthreads_or(kHalf && mine.unit != 0.0f) != 0;
  if (group) return;
  Sums all = sums[0][q];
  if (kHalf && units) {
#pragma unroll 1
    for (int i = 1; i < kGroups; ++i)
      all.join(sums[i][q].top, sums[i][q].sum, sums[i][q].unit, sums[i][q].o);
  } else {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
      const Sums &x = sums[i][q];
      const float to = fmaxf(all.top, x.top);
      all.rescale(to);
      all.add(x.sum, x.o, exp2_(x.top - to));
    }
  }
  put_row<kHd, kBf16, kHalf>(P, all, b, mt, h * P.group + row - mt * P.group, q);
}

// CTAs of a call: at most one share each for the longest that the table holds.
template <class Z>
int grid_of(int B, int M, int group, int kvh, int R, long long room) {
  const long long nrt = (M * group + 8 * R - 1) / (8 * R);
  const long long most = (long long)units_of<Z>((int)room) * nrt * kvh * B;
  const int all = kSms * Z::kCtas;
  return (int)(most < all ? most : all);
}

template <int kHd, int kKind, bool kBf16, int R>
cudaError_t go(const AttnArgs &P, cudaStream_t stream) {
  using Z = Sizes<kHd, kKind, R>;
  using Sh = Shared<kHd, kKind, kBf16, R>;
  static_assert(Sh::kBytes * Z::kCtas <= 227 * 1024 - 1024 * (Z::kCtas - 1), "shared memory");
  static_assert(Z::kCtas <= (kHd > 64 && R > 1 ? 1 : 2), "parts of the workspace");
  static_assert(Z::kSlots >= 3 && 32 * Z::kStage <= Z::kSlot, "rings");
  const int grid = grid_of<Z>(P.B, P.M, P.group, P.c.kvh, R,
                                       (long long)P.cols << P.c.page_shift);
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
  // Joins: by items where each has eight CTAs or more (one sequence of 4099 x 4
  // heads of 256: 9.3 us, 11.4 by CTAs), by CTAs otherwise (64 sequences x 8 heads:
  // 93 us, 96.5 by items).
  const long long heads = (long long)P.B * P.c.kvh;
  cfg.dynamicSmemBytes = 0;
  if (P.B <= 32 && grid >= 8 * heads) {
    cfg.gridDim = dim3((unsigned)(heads * P.M * P.group));
    cfg.blockDim = dim3(512);
    return cudaLaunchKernelEx(&cfg, attn_join_few_kernel<kHd, kKind, kBf16, R>, P, grid);
  }
  const int rows = P.M * P.group < 8 * R ? P.M * P.group : 8 * R;
  constexpr int kRowsBlock = kThreads / (kHd / 4);
  cfg.gridDim = dim3((unsigned)grid, (unsigned)((rows + kRowsBlock - 1) / kRowsBlock));
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<kHd, kKind != kKvBf16, kBf16, R>, P);
}

// Row tiles of 8, 16 or (8 bits, teams) 24: the fewest eights of rows, and of two
// ways with as many the one with fewer passes over the cache.
inline int tile_rows(int kind, int hd, int M, int group) {
  const long long rows = (long long)M * group;
  if (rows <= 8) return 1;
  const bool three = hd == 128 || (hd == 256 && kind != kKvBf16);
  return three && (rows + 23) / 24 * 3 <= (rows + 15) / 16 * 2 ? 3 : 2;
}

template <int kHd, int kKind, int R>
cudaError_t by_type(const AttnArgs &P, bool bf16, cudaStream_t stream) {
  return bf16 ? go<kHd, kKind, true, R>(P, stream) : go<kHd, kKind, false, R>(P, stream);
}

template <int kHd, int kKind>
cudaError_t by_rows(const AttnArgs &P, bool bf16, cudaStream_t stream) {
  const int R = tile_rows(kKind, kHd, P.M, P.group);
  if (R == 1) return by_type<kHd, kKind, 1>(P, bf16, stream);
  if constexpr (kHd == 128 || (kHd == 256 && kKind != kKvBf16)) {
    if (R == 3) return by_type<kHd, kKind, 3>(P, bf16, stream);
  }
  return by_type<kHd, kKind, 2>(P, bf16, stream);
}

template <int kHd>
cudaError_t launch(const AttnArgs &P, bool bf16, cudaStream_t stream) {
  return P.c.kind == kKvBf16   ? by_rows<kHd, kKvBf16>(P, bf16, stream)
         : P.c.kind == kKvInt8 ? by_rows<kHd, kKvInt8>(P, bf16, stream)
                               : by_rows<kHd, kKvE4m3>(P, bf16, stream);
}

// Bytes of the items' ends and the parts: one and two for each CTA, of which an SM
// has at most two.
inline size_t bytes(int kind, int M, int group, int hd) {
  const int R = tile_rows(kind, hd, M, group);
  const int ctas = kSms * (hd > 64 && R > 1 ? 1 : 2);
  return kSplitBytes + (size_t)ctas * 2 * (8 * R) * (hd + 4) * 4;
}

}  // namespace attn

cudaError_t launch_attn_64(const AttnArgs &P, bool bf16, cudaStream_t stream);
cudaError_t launch_attn_128(const AttnArgs &P, bool bf16, cudaStream_t stream);
cudaError_t launch_attn_256(const AttnArgs &P, bool bf16, cudaStream_t stream);

}  // namespace gdn
