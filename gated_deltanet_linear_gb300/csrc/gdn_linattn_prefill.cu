// Chunked linear attention with a decay for each head on tcgen05 tensor cores
// (whole prompts).
//
// The recurrence S_t = a_t S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t taken in
// chunks of C = 64 tokens.  With Gamma_t the sum of g over the chunk's tokens
// up to t and S0 the state before the chunk:
//   o_t  = scale (e^{Gamma_t} S0^T q_t + sum_{s<=t} e^{Gamma_t - Gamma_s} (q_t.k_s) v_s)
//   S_C  = e^{Gamma_C} S0 + sum_t e^{Gamma_C - Gamma_t} k_t v_t^T
// Four products per chunk (D = M x N accumulator in TMEM, lanes = M):
//   QK  [K; Q] K^T               G, rows of Q in lanes 64-127   (A, B smem)
//   QS  S0^T Q^T      [dv][t]    A = S0^T in TMEM, B = Q
//   KV  (V^T f) K     [dv][dk]   A in TMEM, B = K (MN-major)
//   PV  V^T P^T       [dv][t]    A = V^T in TMEM, B = P
// Everything indexed by a value column dv sits in that TMEM lane, so the
// thread of a lane makes its operands and keeps its part of the state.
//
// Precision.  Operands are fp16 numbers scaled by powers of two; with fp32
// rows each operand is hi + lo (22 bits), a product hi hi + hi lo + lo hi,
// accumulated in fp32, so results are fp32 results (a bf16 split keeps 16
// bits).  The products with a lo come first: the accumulation truncates, and
// only the hi hi steps, a third of all, then do so at the size of the sum.  With
// bf16 rows q, k and v fit one fp16 each; the scores, the state and the decayed
// values are hi + lo as with fp32 rows, so o is rounded once (with single fp16
// scores and states it was 9e-4 in norm from the rounded fp32 result, now 3e-5;
// 8 prompts of 4096 tokens took 528 us, and 588 with the second parts).
// The scales: q and k by row, v, the decayed values and the state by column dv
// (the TMEM lane), chosen so that the largest element lies in [2^14, 2^15);
// elements down to 2^-17 of it keep all their bits.  The scores of row t are
// scaled by a bound of the largest |q_t| |k_s| e^{Gamma_t - Gamma_s}, s <= t, over
// the rows that are not zeros, so strong decays and rows of very different
// sizes leave them their bits.  The decayed values' factors are bounded by the
// largest of such rows; their columns take the values' scale where their
// largest is within 2^-17 of it all the same (told by the factors and the
// last 8 rows), else one of their own.  (Always their own took 655 us where
// this takes 610, bf16.)  The state is kept in fp32 registers: a chunk's KV
// product is read out, unscaled and added, so scales may differ from chunk to
// chunk.  Gamma is summed as two floats (48 bits), so strong decays keep the
// small differences between near tokens.
//
// Roles (20 warps, one CTA per SM, persistent over (sequence, head, segment)
// units): 8 warps A hold the state and make its operand and the two V
// operands (the next chunk's V maxima under this one's KV product); 8 warps B
// turn the staged q and k rows into operands in place, make P from G, and the
// output from QS and PV; one warp issues the products,
// one copies rows by TMA (a chunk ahead), two compute the decay vectors.
// All meet through mbarriers; the chunks of successive units form one
// sequence, so a unit's first loads run under the previous one's last chunk.
//
// Few heads: a sequence is cut into segments (see plan()); a first pass
// of the same kernel computes each segment's own contribution to the state
// (KV only), a second kernel chains them into every segment's start state, and
// the main pass runs over all segments at once.
//
// Measured (8 prompts of 4096 tokens, 16 / 48 heads): fp32 690 us (2.20 GB,
// 48 % of the copy rate), bf16 610 us (1.13 GB, 28 %); 33 prompts of up to 111
// tokens, fp32 92 us, bf16 85; one of 32701 tokens, 2 / 8 heads, bf16 140 us, fp32
// 158.  Bound by the latency of each chunk's chain (rows - decay vectors - V
// operands - KV - state, and scores - P - PV - output) on 4 to 5 warps a
// scheduler: fp32 issues in 56 % of the cycles, the tensor cores are busy in
// 34 %, DRAM 38 %; bf16 61, 21 and 21 %.  The code of all roles together is more
// than the instruction cache bears (15 % of its requests miss): more unrolling,
// or warps for more roles, cost more than they hid (24 and 32 warps with packed
// arithmetic 9000 cycles a chunk where 20 took 7000; the score loop unrolled
// +12 %), 1.4 KB less of it gave 5 %.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "gdn_internal.cuh"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"
#include "gdn_vec.cuh"

namespace gdn {

__device__ unsigned int g_linattn_timeouts = 0;

namespace {

using namespace tc;

constexpr int kC = 64, kD = kDim;
constexpr int kGroup = 256;               // threads of group A and of group B
constexpr int kIssuer = 16, kLoader = 17, kGates = 18;
constexpr int kThreads = 640;
constexpr int kSms = 152;
constexpr uint32_t kWaitLimit = 1u << 24;

// Shared memory (bytes from a 1024-aligned base).  The q, k regions hold a
// chunk's staged rows (K then Q), converted in place to the [K; Q] operand of
// 128 rows x 128 fp16: the rows of a group of 8 stay in the bytes that they
// were staged in, as 128-byte-swizzled blocks of 8 rows x 64 columns (hi
// columns 0-63, hi 64-127, then the same of lo), so a warp converts a group by
// itself.
constexpr uint32_t OFF_KQ = 0, kKQ = 65536;   // by chunk parity
constexpr uint32_t OFF_V = 131072, kV = 32768;  // staged v rows, by parity
constexpr uint32_t OFF_P = 196608;            // P operand 64 x 64, hi, lo
// decay vectors of a chunk, buffer it & 3, 512 floats:
constexpr int VA = 0, VB = 64, VF = 128, VCA = 192, VCB = 256, VGH = 320,
              VGL = 384, VM = 448;
constexpr uint32_t OFF_VEC = 212992;
constexpr uint32_t OFF_EXP = OFF_VEC + 4 * 2048;    // row exponents [2][128]
constexpr uint32_t OFF_LANE = OFF_EXP + 2 * 512;    // column factors [2][2][128]
constexpr uint32_t OFF_PV = OFF_LANE + 2 * 1024;    // exchange: V maxima [2][2][128]
constexpr uint32_t OFF_PS = OFF_PV + 2048;          // exchange: state maxima
constexpr uint32_t OFF_P8 = OFF_PS + 1024;          // V maxima of the last rows [2][128]
constexpr uint32_t OFF_BAD = OFF_P8 + 1024;         // first bad token [4][2][128]
constexpr uint32_t OFF_BAR = OFF_BAD + 1024;
constexpr uint32_t kSmemUsed = OFF_BAR + 256;
constexpr uint32_t kSmemAlloc = kSmemUsed + 1024;   // room to align the base
static_assert(kSmemAlloc <= 232448, "shared memory");

// TMEM columns (512): the KV product, the state operand (hi, lo), the V and
// decayed V operands (hi, lo), QS and G.  PV takes the decayed operand's columns,
// which KV has read, so that the next QK need not wait for the output.
constexpr uint32_t T_D = 0, T_SOP = 128, T_VOP = 256, T_WOP = 320, T_QS = 384,
                   T_G = 448, T_PV = T_WOP;

__host__ __device__ constexpr uint32_t idesc16(int M, int N, int b_mn) {
  // fp16 operands (format 0), fp32 accumulator; B MN-major if b_mn
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// The output's factors by column carry 2^-15 and those by row 2^15, so that a
// product times the first stays below 128 times its column's largest element.
constexpr float kOut = 0x1p-15f;
constexpr int kOutExp = 15;

struct Args {
  float *S;             // [B][vh][128][128], in/out
  float *ws_state;      // [B vh][nseg][128][128]: own sums, then start states
  double *ws_decay;     // [B vh][nseg][2]: log2 of a segment's decay, in two parts
  const float *g;
  void *o;
  const int *lens;
  int *err;
  float scale;
  int g_head, vh, rep, T, nseg, per_seg, units;  // per_seg: chunks of a segment
};

// ------------------------------------------------------------- sequencing

// The chunks this CTA works on, in order; every role walks the same list.
// (next() is written once per role: the code of all roles together should
// stay within the instruction cache.)
template <bool kLocal>
struct Walk {
  const Args *p;
  int u, c, c_hi, it;   // unit, chunk, end of its chunks, running index
  int head, b, vi, seg, n;
  bool ok, first;
  __device__ Walk(const Args &P)
      : p(&P), u((int)blockIdx.x - (int)gridDim.x), c(0), c_hi(0), it(-1), ok(false) {}
  // Decodes unit u; false if its sequence has no valid length.
  __device__ __forceinline__ bool decode() {
    const unsigned per = kLocal ? p->nseg - 1 : p->nseg;
    head = (unsigned)u / per;
    seg = u - head * per;
    b = (unsigned)head / (unsigned)p->vh;
    vi = head - b * p->vh;
    n = p->T;
    if (p->lens) n = __shfl_sync(0xffffffffu, __ldg(p->lens + b), 0);
    const bool good = n >= 0 && n <= p->T;
    if (!good) n = 0;
    c = seg * p->per_seg;
    c_hi = min(c + p->per_seg, (n + kC - 1) / kC);
    return good;
  }
  // The next chunk; false (and !ok) behind the last one.
  __device__ __forceinline__ bool next() {
    ++it;
    first = false;
    ok = true;
    if (++c < c_hi) return true;
    first = true;
#pragma unroll 1
    do {
      u += gridDim.x;
      if (u >= p->units) return ok = false;
      decode();
    } while (c >= c_hi);
    return true;
  }
  __device__ bool last() const { return c + 1 >= c_hi; }
  __device__ int valid() const { return min(kC, n - c * kC); }  // tokens
};

// ------------------------------------------------------------ small pieces

__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __int_as_float((e + 127) << 23);
}

// e with 2^14 <= m 2^e < 2^15, at most 126; NaN and infinities give -114.
__device__ __forceinline__ int scale_exp(float m) {
  return min(141 - (__float_as_int(m) >> 23), 126);
}

// max(|m|, |x|) and max(|m|, |x|, |y|), NaN if any is
__device__ __forceinline__ float amax(float m, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(m)), "f"(fabsf(x)));
  return r;
}
__device__ __forceinline__ float amax(float m, float x, float y) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(x), "f"(y));
  return r;
}

// Unevaluated sum of two floats (about 48 bits): the cumulative log decays.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two add2(Two a, Two b) {
  const float s = a.h + b.h, v = s - a.h;
  const float e = (a.h - (s - v)) + (b.h - v) + (a.l + b.l);
  const float h = s + e;
  return Two{h, e - (h - s)};
}
// 2^x in one instruction (2^-22 relative; 0 where the result is below 2^-126).
// Its arguments are rounded to a float, 2^-24 |x|: less than 2^-24 of the whole for
// weights 2^x <= 1; larger exponents are taken apart into integer and rest.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ Two shfl_up2(Two x, int d) {
  return Two{__shfl_up_sync(0xffffffffu, x.h, d), __shfl_up_sync(0xffffffffu, x.l, d)};
}

// x - h, exactly
__device__ __forceinline__ float less(float x, __half h) {
  float r;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;"
      : "=f"(r)
      : "h"(__half_as_ushort(h)), "h"((unsigned short)0xbc00), "f"(x));
  return r;
}

// The fp16 parts of two floats: hi = fp16(x) and, with kLo, lo = fp16(x - hi).
template <bool kLo>
__device__ __forceinline__ void split2(F2 v, uint32_t &hi, uint32_t &lo) {
  const float2 x = unpack(v);
  const __half2 h = __floats2half2_rn(x.x, x.y);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  if (kLo) {
    const __half2 l = __floats2half2_rn(less(x.x, __low2half(h)), less(x.y, __high2half(h)));
    lo = *reinterpret_cast<const uint32_t *>(&l);
  }
}

// Elements c0 .. c0+15 of this lane of an A operand in TMEM.
template <bool kLo>
__device__ __forceinline__ void put16(uint32_t hi, uint32_t lo, int c0, const F2 *x) {
  uint32_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split2<kLo>(x[i], h[i], l[i]);
  tmem_st8_async(hi + (uint32_t)(c0 >> 1), h);
  if (kLo) tmem_st8_async(lo + (uint32_t)(c0 >> 1), l);
}

// 16 TMEM columns of this thread's lane, as 8 pairs; tmem_wait_ld before use.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&u)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]),
        "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]),
        "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(taddr));
}

template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&u)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // the loaded registers are defined only from here on
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(u[i]));
}

__device__ __forceinline__ F2 pair(const uint32_t *u) {
  return pack(__uint_as_float(u[0]), __uint_as_float(u[1]));
}

__device__ __forceinline__ void mbar_arrive(uint32_t mbar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(mbar) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t mbar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mbar),
               "r"(bytes)
               : "memory");
}

// Waits for the phase of this parity; gives up after kWaitLimit polls, or as
// soon as another role of the CTA has (the flag): every role then runs on to
// the end, through the same barriers, without waiting again.
__device__ __forceinline__ void wait_bar(uint32_t bar, uint32_t parity, volatile int *fail) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return;
    if (*fail) return;
  }
  *fail = 1;
}

// A warp's part of "operands ready" (one arrival per warp; 256 arrivals on one
// barrier took longer than the work they announced): its TMEM accesses
// ordered, and with kSmem its shared-memory writes made visible to the tensor
// cores.
template <bool kSmem>
__device__ __forceinline__ void signal_ready(uint32_t mbar) {
  if (kSmem) fence_proxy_async();
  fence_before_sync();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(mbar);
}

// Where every role ends: after it nothing of the CTA is in flight.
__device__ __forceinline__ void cta_end() {
  fence_before_sync();
  asm volatile("bar.sync 0, %0;" ::"n"(kThreads) : "memory");
  fence_after_sync();
}

__device__ __forceinline__ void bar_pair(int quad) {  // warps w and w + 4 of A
  asm volatile("bar.sync %0, 64;" ::"r"(quad + 1) : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t smem, const CUtensorMap *map, int h,
                                         int t0, int b, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(h), "r"(t0), "r"(b), "r"(mbar)
      : "memory");
}

// ---------------------------------------------------------------- products

// Descriptors: the high word holds the stride between 8-row groups, the low
// word the address (and, MN-major, the distance of 64-column blocks), so the
// steps of a product are additions to the low word.
__device__ __forceinline__ uint32_t desc_hi(uint32_t stride) {
  return (uint32_t)(desc_sw128(0) >> 32) & ~0x3FFFu | (stride >> 4);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc64(uint32_t hi, uint32_t lo) {
  return ((uint64_t)hi << 32) | lo;
}
// Bytes of K step ks (16 elements) from a K-major operand's start.
__host__ __device__ constexpr uint32_t kstep(int ks) {
  return (uint32_t)((ks >> 2) * 1024 + (ks & 3) * 32);
}

// ------------------------------------------------------------ row operands

// A group of 8 staged rows (8 x 512 bytes fp32, or 256 bf16) on its way to the
// fp16 operand in the same bytes, by one warp: lane l has rows 2 i + (l >> 4)
// and of each, with m = l & 15, columns 4 m .. + 3 and 64 + 4 m .. + 3 (fp32) or
// 8 m .. + 7 (bf16), so that every access of a quarter warp covers whole banks.
template <bool kBf16>
struct RowGroup {
  static constexpr uint32_t kRow = kBf16 ? 256 : 512;
  static constexpr int kN = kBf16 ? 4 : 8;
  uint32_t x[4][kN];  // as staged
  __device__ __forceinline__ void read(const unsigned char *g8, int lane) {
    g8 += (lane >> 4) * kRow + (lane & 15) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kN; j += 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(g8 + 2 * i * kRow + 64 * j);
        x[i][j] = u.x;
        x[i][j + 1] = u.y;
        x[i][j + 2] = u.z;
        x[i][j + 3] = u.w;
      }
  }
  // Scale exponents of the rows to ex[8] (127: nothing but zeros).  The four
  // rows of a lane are reduced together, half of them sent on at each step.
  __device__ __forceinline__ void scales(int *ex, int lane) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kBf16) {  // |x| by pairs, as integers: NaN above all
        uint32_t u = x[i][0] & 0x7fff7fffu;
#pragma unroll
        for (int j = 1; j < kN; ++j) u = __vmaxu2(u, x[i][j] & 0x7fff7fffu);
        m[i] = __uint_as_float(max(u << 16, u & 0xffff0000u));
      } else {
        m[i] = 0.f;
#pragma unroll
        for (int j = 0; j < kN; j += 2)
          m[i] = amax(m[i], __uint_as_float(x[i][j]), __uint_as_float(x[i][j + 1]));
      }
    }
    const bool b3 = lane & 8, b2 = lane & 4;
    const float s0 = __shfl_xor_sync(0xffffffffu, b3 ? m[0] : m[2], 8);
    const float s1 = __shfl_xor_sync(0xffffffffu, b3 ? m[1] : m[3], 8);
    const float m0 = amax(b3 ? m[2] : m[0], s0), m1 = amax(b3 ? m[3] : m[1], s1);
    float t = amax(b2 ? m1 : m0, __shfl_xor_sync(0xffffffffu, b2 ? m0 : m1, 4));
    t = amax(t, __shfl_xor_sync(0xffffffffu, t, 2));
    t = amax(t, __shfl_xor_sync(0xffffffffu, t, 1));
    if ((lane & 3) == 0)
      ex[(lane >> 1 & 6) + (lane >> 4)] = t == 0.f ? 127 : scale_exp(t);
  }
  // (behind a __syncwarp: every row of the group is read, the exponents written)
  __device__ __forceinline__ void write(unsigned char *g8, const int *ex, int lane) {
    const int m16 = lane & 15, r1 = lane >> 4;
    ex += r1;
    g8 += r1 * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sc = pow2(ex[2 * i]);
      const F2 f = pack(sc, sc);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 v = kBf16 ? pack(__uint_as_float(x[i][j] << 16),
                                  __uint_as_float(x[i][j] & 0xffff0000u))
                           : pair(&x[i][kBf16 ? 0 : 2 * j]);
        split2<!kBf16>(mul2(v, f), hi[j], lo[j]);
      }
      // row r = 2 i + r1: blocks of 16 bytes at their place XOR r
      if (kBf16) {
        *reinterpret_cast<uint4 *>(g8 + (m16 >> 3) * 1024 + i * 256 +
                                   ((((m16 & 7) ^ r1) << 4) ^ (i << 5))) =
            make_uint4(hi[0], hi[1], hi[2], hi[3]);
      } else {
        unsigned char *p = g8 + i * 256 + ((((m16 >> 1) ^ r1) << 4) ^ (i << 5)) + (m16 & 1) * 8;
        *reinterpret_cast<uint2 *>(p) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2 *>(p + 1 * 1024) = make_uint2(hi[2], hi[3]);
        *reinterpret_cast<uint2 *>(p + 2 * 1024) = make_uint2(lo[0], lo[1]);
        *reinterpret_cast<uint2 *>(p + 3 * 1024) = make_uint2(lo[2], lo[3]);
      }
    }
  }
};

// ------------------------------------------------------------------ kernel

template <bool kBf16, bool kLocal>
__global__ void __launch_bounds__(kThreads, 1)
    linattn_chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ Args P) {
  constexpr bool kLo = !kBf16;                 // second parts of q, k, v
  constexpr uint32_t kRow = kBf16 ? 256 : 512; // bytes of a token row
  constexpr uint32_t kGrp = 8 * kRow;          // of 8 rows, staged or converted
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_s = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t sb = (raw_s + 1023u) & ~1023u;
  unsigned char *gb = smem_raw + (sb - raw_s);
  const uint32_t bar0 = sb + OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  // rows landed / region free again / operand made, by chunk parity
  const uint32_t staged = bar(0), kq_free = bar(2), rdy_kq = bar(4);
  const uint32_t vstaged = bar(6), v_free = bar(8);
  const uint32_t rdy_s = bar(10), rdy_v = bar(11), rdy_p = bar(12);
  const uint32_t done_qk = bar(13), done_o = bar(14), done_kv = bar(15);
  const uint32_t acc_free = bar(16), drain = bar(17), vecs = bar(18);  // 18..21
  volatile uint32_t *slot = reinterpret_cast<volatile uint32_t *>(gb + OFF_BAR + 184);
  volatile int *fail = reinterpret_cast<volatile int *>(gb + OFF_BAR + 188);
  auto vec = [&](int it) { return reinterpret_cast<float *>(gb + OFF_VEC + (it & 3) * 2048); };
  auto rowexp = [&](int it) { return reinterpret_cast<int *>(gb + OFF_EXP + (it & 1) * 512); };
  auto lanef = [&](int it) { return reinterpret_cast<float *>(gb + OFF_LANE + (it & 1) * 1024); };

  // first token of a chunk whose v is not finite, by half and column
  auto badtok = [&](int it) {
    return reinterpret_cast<unsigned char *>(gb + OFF_BAD + (it & 3) * 256);
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, half = (warp >> 2) & 1;
  const int myrow = 32 * quad + lane;          // TMEM lane

  if (warp == kIssuer) tmem_alloc(sb + OFF_BAR + 184, 512);
  if (tid == 0) {
    // one arrival each, or one from each warp of a group
    constexpr uint32_t kByWarps = 0x3u << 4 | 0x1fu << 8 | 1u << 16;
#pragma unroll 1
    for (int i = 0; i < 22; ++i) mbar_init(bar(i), (kByWarps >> i & 1) ? kGroup / 32 : 1);
    *fail = 0;
  }
  // behind the kernel before it: nothing is read or written before it has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);

  // Registers: launched with 640 x 96 = 61,440; 256 x 120 + 256 x 88 + 128 x 56
  // = 60,416 after the split.  No code follows the roles' branches: it would
  // have to fit the smallest count.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    // ============================================ group A: state, V operands
    F2 s[kC / 2];  // state rows dk = 64 half .. + 63 of column dv = myrow
    float *ps = reinterpret_cast<float *>(gb + OFF_PS);
    auto px = [&](int it) { return reinterpret_cast<float *>(gb + OFF_PV + (it & 1) * 1024); };
    auto p8 = [&](int it) { return reinterpret_cast<float *>(gb + OFF_P8 + (it & 1) * 512); };
    // this thread's 32 v values of a chunk: column myrow of rows 32 half ..
    auto vcol = [&](int it) {
      return gb + OFF_V + (it & 1) * kV + 32 * half * kRow + myrow * (kRow / kD);
    };
    auto vload = [&](const unsigned char *vp, int t) -> F2 {  // tokens t and t + 1
      if (kBf16)
        return pack(__uint_as_float((uint32_t) * reinterpret_cast<const unsigned short *>(
                                        vp + t * kRow) << 16),
                    __uint_as_float((uint32_t) * reinterpret_cast<const unsigned short *>(
                                        vp + (t + 1) * kRow) << 16));
      return pack(*reinterpret_cast<const float *>(vp + t * kRow),
                  *reinterpret_cast<const float *>(vp + (t + 1) * kRow));
    };
    // The largest |v| of chunk `it` (and of its last 8 rows) and what is not finite,
    // to the exchange.
    auto v_max = [&](int it, int valid) {
      wait_bar(vstaged + 8 * (it & 1), (it >> 1) & 1, fail);
      unsigned char *vp = vcol(it);
      const int nv = valid - 32 * half;
      if (nv < 32) {  // rows behind the end are zeros, whatever they hold
#pragma unroll 1
        for (int t = max(nv, 0); t < 32; ++t) {
          if (kBf16)
            *reinterpret_cast<unsigned short *>(vp + t * kRow) = 0;
          else
            *reinterpret_cast<float *>(vp + t * kRow) = 0.f;
        }
        fence_proxy_async();  // the copy engine writes these bytes next
      }
      float m = 0.f, m8;
#pragma unroll 1
      for (int t0 = 0; t0 < 32; t0 += 8) {
        m8 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 f = unpack(vload(vp, t0 + j));
          m8 = amax(m8, f.x, f.y);
        }
        m = amax(m, m8);
      }
      if (half) p8(it)[myrow] = m8;
      // A value that is not finite must not reach the rows before it (its
      // weight there is 0, but 0 * inf is NaN): PV takes 0 for it, and the
      // output becomes NaN from its token on.
      int bad = kC;
      if (!isfinite(m)) {
        m = 0.f;
#pragma unroll 1
        for (int t = 30; t >= 0; t -= 2) {
          const float2 f = unpack(vload(vp, t));
          if (isfinite(f.y)) m = amax(m, f.y); else bad = 32 * half + t + 1;
          if (isfinite(f.x)) m = amax(m, f.x); else bad = 32 * half + t;
        }
      }
      px(it)[128 * half + myrow] = m;
      badtok(it)[128 * half + myrow] = bad;
    };
    // units without a chunk of their own: their states, and bad lengths
    if (P.lens || kLocal || P.nseg > 1) {
      Walk<kLocal> w(P);
      for (int u = blockIdx.x; u < P.units; u += gridDim.x) {
        w.u = u;
        const bool good = w.decode();
        if (!good && tid == 0 && w.seg == 0 && w.vi == 0 && P.err) *P.err = 1;
        if (w.c < w.c_hi) continue;
        const size_t at = ((size_t)w.head * P.nseg + w.seg) * kD * kD;
        if (kLocal) {
          for (int j = 0; j < kC; ++j)
            P.ws_state[at + (size_t)(kC * half + j) * kD + myrow] = 0.f;
        } else if (good && P.nseg > 1 && w.seg == P.nseg - 1) {
          for (int j = 0; j < kC; ++j) {
            const size_t e = (size_t)(kC * half + j) * kD + myrow;
            P.S[(size_t)w.head * kD * kD + e] = P.ws_state[at + e];
          }
        }
      }
    }
    Walk<kLocal> w(P);
    if (w.next()) v_max(0, w.valid());
    while (w.ok) {
      const int it = w.it, head = w.head, seg = w.seg;
      const bool last = w.last();
      if (w.first) {
        const size_t at = ((size_t)head * P.nseg + seg) * kD * kD;
        const float *src = (P.nseg > 1 ? P.ws_state + at : P.S + at) + kC * half * kD + myrow;
#pragma unroll
        for (int j = 0; j < kC; j += 2)
          s[j / 2] = kLocal ? 0ull : pack(src[j * kD], src[(j + 1) * kD]);
      }
      if (!kLocal) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < kC / 2; ++j) {
          const float2 x = unpack(s[j]);
          m = amax(m, x.x, x.y);
        }
        ps[128 * half + myrow] = m;
      }
      // (one exchange a chunk: both halves' v maxima, made under the last
      // chunk's KV product, and state maxima)
      bar_pair(quad);
      if (!kLocal) {
        // ---- the state operand
        const int e = scale_exp(amax(ps[myrow], ps[128 + myrow]));
        const F2 f = pack(pow2(e), pow2(e));
#pragma unroll
        for (int c0 = 0; c0 < kC; c0 += 16) {
          F2 x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = mul2(s[c0 / 2 + j], f);
          put16<true>(tl + T_SOP, tl + T_SOP + 64, 64 * half + c0, x);
        }
        if (half == 0) lanef(it)[myrow] = pow2(-e) * kOut;
        tmem_wait_st();
        signal_ready<false>(rdy_s);
      }
      // ---- V^T and (V f)^T operands, lane dv, K = t = 32 half .. + 31
      const float vmax = amax(px(it)[myrow], px(it)[128 + myrow]);
      const int ea = scale_exp(vmax);
      wait_bar(vecs + 8 * (it & 3), (it >> 2) & 1, fail);
      const unsigned char *vp = vcol(it);
      // Whether the decayed values need a scale of their own: some rows count for
      // less than 2^-17 of others (strong decays, key rows of zeros or of very
      // different sizes) and a column's last 8 values do not outweigh that.
      const bool need = __any_sync(0xffffffffu, p8(it)[myrow] * vec(it)[VM + 3] < vmax);
      int ew = ea;
      const float gC = vec(it)[VM];
      float inv;
      {
        const F2 fa = pack(pow2(ea), pow2(ea));
        if (!kLocal) {
          // V's columns are free once the previous chunk's PV has read them, the
          // decayed ones once the output has been made of it
          if (it > 0) wait_bar(acc_free, (it - 1) & 1, fail);
          fence_after_sync();
          if (half == 0) lanef(it)[128 + myrow] = pow2(-ea) * kOut;
        }
        const bool any_bad =
            !kLocal && __any_sync(0xffffffffu, badtok(it)[128 * half + myrow] < kC);
#pragma unroll 1
        for (int t0 = 0; t0 < 32; t0 += 16) {
          const F2 *vf = reinterpret_cast<const F2 *>(vec(it) + VF + 32 * half + t0);
          F2 x[8], y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = mul2(vload(vp, t0 + 2 * j), fa);
            y[j] = mul2(x[j], vf[j]);
          }
          put16<true>(tl + T_WOP, tl + T_WOP + 32, 32 * half + t0, y);
          if (!kLocal) {
            if (any_bad)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 f = unpack(x[j]);
                x[j] = pack(isfinite(f.x) ? f.x : 0.f, isfinite(f.y) ? f.y : 0.f);
              }
            put16<kLo>(tl + T_VOP, tl + T_VOP + 32, 32 * half + t0, x);
          }
        }
        if (__builtin_expect(need, 0)) {
          // The decayed values once more, scaled by their own largest, lest fp16
          // take their bits (or all of them: where v or k are zeros in the rows that
          // weigh most, the others are the whole state).  Both halves go through
          // all 64 rows: a barrier here would be passed by some warps alone where a
          // wait has run out.
          const F2 *vf = reinterpret_cast<const F2 *>(vec(it) + VF);
          const unsigned char *v0 = vp - 32 * half * kRow;
          float m = 0.f;
#pragma unroll 2
          for (int t = 0; t < kC; t += 2) {
            const float2 y = unpack(mul2(vload(v0, t), vf[t / 2]));
            m = amax(m, y.x, y.y);
          }
          ew = scale_exp(m);
          vf += 16 * half;
          const F2 fw = pack(pow2(ew), pow2(ew));
#pragma unroll 1
          for (int t0 = 0; t0 < 32; t0 += 16) {
            F2 y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)  // (in this order: no step leaves the floats)
              y[j] = mul2(mul2(vload(vp, t0 + 2 * j), vf[t0 / 2 + j]), fw);
            put16<true>(tl + T_WOP, tl + T_WOP + 32, 32 * half + t0, y);
          }
        }
        inv = pow2(-ew) * vec(it)[VM + 2];
        tmem_wait_st();
        signal_ready<false>(rdy_v);
        if (lane == 0) mbar_arrive(v_free + 8 * (it & 1));
      }
      // ---- the next chunk's v maxima, under this one's product
      if (w.next()) v_max(w.it, w.valid());
      // ---- the state after the chunk
      wait_bar(done_kv, it & 1, fail);
      fence_after_sync();
      const F2 a1 = pack(inv, inv), a2 = pack(gC, gC);
#pragma unroll
      for (int c0 = 0; c0 < kC; c0 += 16) {
        uint32_t d[16];
        tmem_ld16_async(tl + T_D + 64 * half + c0, d);
        tmem_wait_ld(d);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          s[c0 / 2 + j] = fma2(pair(d + 2 * j), a1, mul2(s[c0 / 2 + j], a2));
      }
      if (kLocal) signal_ready<false>(rdy_s);  // the KV columns are read
      if (last && (kLocal || seg == P.nseg - 1)) {
        float *dst = (kLocal ? P.ws_state + ((size_t)head * P.nseg + seg) * kD * kD
                             : P.S + (size_t)head * kD * kD) +
                     kC * half * kD + myrow;
#pragma unroll
        for (int j = 0; j < kC; j += 2) {
          const float2 x = unpack(s[j / 2]);
          dst[j * kD] = x.x;
          dst[(j + 1) * kD] = x.y;
        }
      }
    }
    cta_end();
    if (*fail) {
      // a wait ran out: everything this CTA was to write becomes NaN, so the
      // failure shows in the results as well as in the counter
      if (tid == 0) atomicAdd(&g_linattn_timeouts, 1u);
      const float nan = __int_as_float(0x7fffffff);
      Walk<kLocal> f(P);
#pragma unroll 1
      for (f.u = blockIdx.x; f.u < P.units; f.u += gridDim.x) {
        f.decode();
        float *dst = kLocal ? P.ws_state + ((size_t)f.head * P.nseg + f.seg) * kD * kD
                            : P.S + (size_t)f.head * kD * kD;
#pragma unroll 1
        for (int e = tid; e < kD * kD; e += kGroup) dst[e] = nan;
        const int t_end = kLocal ? 0 : min(f.n, f.c_hi * kC);
#pragma unroll 1
        for (int t = f.c * kC; t < t_end; ++t) {
          const size_t row = (((size_t)f.b * P.T + t) * P.vh + f.vi) * kRow;
          if (tid < (int)kRow / 4)
            *reinterpret_cast<uint32_t *>(static_cast<unsigned char *>(P.o) + row + 4 * tid) =
                0x7fffffffu;
        }
      }
    }
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    // ======================================= group B: q, k rows, P, output
    Walk<kLocal> w(P), nx(P);  // the chunk at hand (none at first), the next
    for (bool more = true; more;) {
      w = nx;
      more = nx.next();
      const int it = w.it;
      const float *vc = vec(it);
      if (!kLocal && w.ok) {
      // ---- P[t][s] = G e^{Gamma_t - Gamma_s}, s <= t (lanes 64-127: q rows)
      wait_bar(vecs + 8 * (it & 3), (it >> 2) & 1, fail);
      wait_bar(done_qk, it & 1, fail);
      fence_after_sync();
      if (quad >= 2) {
        const int t = myrow - kC;
        const float at = vc[VA + t];
        const bool fac = vc[VM + 1] != 0.f;
        unsigned char *pr = gb + OFF_P + t * 128;
        const F2 at2 = pack(at, at);
#pragma unroll 1
        for (int s0 = 32 * half; s0 < 32 * half + 32; s0 += 16) {
          F2 x[8];
          if (s0 < 32 * (quad - 1)) {  // some s <= t in this warp
            uint32_t r[16];
            tmem_ld16_async(tl + T_G + s0, r);
            tmem_wait_ld(r);
            const F2 *vb = reinterpret_cast<const F2 *>(vc + VB + s0);
            if (fac) {
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = mul2(pair(r + 2 * j), mul2(at2, vb[j]));
            } else {
              const float *h = vc + VGH + s0, *l = vc + VGL + s0;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 n = unpack(vb[j]);
                x[j] = mul2(pair(r + 2 * j),
                            pack(ex2(((at - h[2 * j]) - l[2 * j]) + n.x),
                                 ex2(((at - h[2 * j + 1]) - l[2 * j + 1]) + n.y)));
              }
            }
            if (s0 + 15 > 32 * (quad - 2))
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 f = unpack(x[j]);
                x[j] = pack(s0 + 2 * j <= t ? f.x : 0.f, s0 + 2 * j + 1 <= t ? f.y : 0.f);
              }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0ull;
          }
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) split2<true>(x[j], hi[j], lo[j]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            unsigned char *p = pr + ((((s0 >> 3) + c) ^ (t & 7)) << 4);
            *reinterpret_cast<uint4 *>(p) =
                make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
            *reinterpret_cast<uint4 *>(p + 8192) =
                make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
          }
        }
      }
      signal_ready<true>(rdy_p);
      }
      // ---- the next chunk's rows, under this one's products: two groups of 8 a
      // warp (the state pass takes the k rows alone)
      if (more) {
        const int par = nx.it & 1;
        wait_bar(staged + 8 * par, (nx.it >> 1) & 1, fail);
#pragma unroll 1
        for (int grp = warp - 8; grp < (kLocal ? 8 : 16); grp += 8) {
          unsigned char *g8 = gb + OFF_KQ + par * kKQ + grp * kGrp;
          const int nr = nx.valid() - 8 * (grp & 7);
          if (nr < 8) {  // rows behind the end are zeros, whatever they hold
#pragma unroll 1
            for (uint32_t at = max(nr, 0) * kRow + 16 * lane; at < kGrp; at += 512)
              *reinterpret_cast<uint4 *>(g8 + at) = make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
          }
          int *ex = rowexp(nx.it) + 8 * grp;
          RowGroup<kBf16> g;
          g.read(g8, lane);
          g.scales(ex, lane);
          __syncwarp();
          g.write(g8, ex, lane);
        }
        signal_ready<true>(rdy_kq + 8 * par);
      }
      if (kLocal || !w.ok) continue;
      // ---- o^T = cA QS + cB PV, lane dv, columns t = 32 half .. + 31: a warp
      // stores 32 columns of a row at a time, straight to the output
      wait_bar(done_o, it & 1, fail);
      fence_after_sync();
      const float fs = lanef(it)[myrow], fv = lanef(it)[128 + myrow];
      const int nv = w.valid() - 32 * half;
      typedef typename std::conditional<kBf16, __nv_bfloat16, float>::type Out;
      const size_t pitch = (size_t)P.vh * kD;
      Out *op = static_cast<Out *>(P.o) +
                ((size_t)w.b * P.T + (size_t)w.c * kC + 32 * half) * pitch + w.vi * kD + myrow;
      const F2 fs2 = pack(fs, fs), fv2 = pack(fv, fv);
      const int bad = min((int)badtok(it)[myrow], (int)badtok(it)[128 + myrow]) - 32 * half;
      Out *p = op;
#pragma unroll 1
      for (int t0 = 0; t0 < 32; t0 += 16) {
        uint32_t qs[16], pv[16];
        tmem_ld16_async(tl + T_QS + 32 * half + t0, qs);
        tmem_ld16_async(tl + T_PV + 32 * half + t0, pv);
        tmem_wait_ld(qs);
        tmem_wait_ld(pv);
        if (t0 == 16) signal_ready<false>(acc_free);
        const F2 *ca = reinterpret_cast<const F2 *>(vc + VCA + 32 * half + t0);
        const F2 *cb = reinterpret_cast<const F2 *>(vc + VCB + 32 * half + t0);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 y = unpack(fma2(mul2(pair(qs + j), fs2), ca[j / 2],
                                       mul2(mul2(pair(pv + j), fv2), cb[j / 2])));
          if (j < nv - t0) *p = (Out)y.x;
          p += pitch;
          if (j + 1 < nv - t0) *p = (Out)y.y;
          p += pitch;
        }
      }
      // (the same thread's stores, so in order)
#pragma unroll 1
      for (int j = max(bad, 0); j < min(nv, 32); ++j)
        op[j * pitch] = (Out)__int_as_float(0x7fffffff);
    }
    cta_end();
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == kIssuer) {
    // ===================================================== the issuing warp
    {
      const uint32_t one = elect();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t idn = idesc16(128, kC, 0), idk = idesc16(128, kD, 1);
      const uint32_t hi = desc_hi(kGrp), hi_p = desc_hi(1024);
      const uint32_t lo_p = desc_lo(sb + OFF_P, 16);
      for (Walk<kLocal> w(P); w.next();) {
        const int it = w.it;
        const uint32_t kq = sb + OFF_KQ + (it & 1) * kKQ;
        wait_bar(rdy_kq + 8 * (it & 1), (it >> 1) & 1, fail);
        if (!kLocal) {
          // (G is free: P of the last chunk is made)
          fence_after_sync();
          const uint32_t lo_k = desc_lo(kq, 16), lo_q = lo_k + (8 * kGrp >> 4);
          if (kLo)
#pragma unroll 1
            for (int ks = 0; ks < kD / 16; ++ks) {
              const uint64_t h = desc64(hi, lo_k + (kstep(ks) >> 4));
              const uint64_t l = desc64(hi, lo_k + ((kstep(ks) + 2048) >> 4));
              mma_ss(one, tm + T_G, h, l, idn, ks > 0);
              mma_ss(one, tm + T_G, l, h, idn, 1u);
            }
#pragma unroll 1
          for (int ks = 0; ks < kD / 16; ++ks) {
            const uint64_t h = desc64(hi, lo_k + (kstep(ks) >> 4));
            mma_ss(one, tm + T_G, h, h, idn, kLo || ks > 0);
          }
          commit_one(one, done_qk);
          wait_bar(rdy_s, it & 1, fail);
          if (it > 0) wait_bar(acc_free, (it - 1) & 1, fail);
          fence_after_sync();
#pragma unroll 1
          for (int ks = 0; ks < kD / 16; ++ks) {
            const uint32_t a = tm + T_SOP + 8u * ks;
            mma_ts(one, tm + T_QS, a + 64u, desc64(hi, lo_q + (kstep(ks) >> 4)), idn, ks > 0);
            if (kLo)
              mma_ts(one, tm + T_QS, a, desc64(hi, lo_q + ((kstep(ks) + 2048) >> 4)), idn, 1u);
          }
#pragma unroll 1
          for (int ks = 0; ks < kD / 16; ++ks)
            mma_ts(one, tm + T_QS, tm + T_SOP + 8u * ks, desc64(hi, lo_q + (kstep(ks) >> 4)), idn,
                   1u);
        } else {
          // the KV columns are free once the state has taken the last product
          if (it > 0) wait_bar(rdy_s, (it - 1) & 1, fail);
        }
        wait_bar(rdy_v, it & 1, fail);
        fence_after_sync();
        {
          const uint32_t lo_k = desc_lo(kq, 1024);  // rows are K: two groups a step
#pragma unroll 1
          for (int ks = 0; ks < kC / 16; ++ks) {
            const uint64_t h = desc64(hi, lo_k + (ks * 2 * kGrp >> 4));
            const uint64_t l = desc64(hi, lo_k + ((ks * 2 * kGrp + 2048) >> 4));
            const uint32_t a = tm + T_WOP + 8u * ks;
            mma_ts(one, tm + T_D, a + 32u, h, idk, ks > 0);
            if (kLo) mma_ts(one, tm + T_D, a, l, idk, 1u);
          }
#pragma unroll 1
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_ts(one, tm + T_D, tm + T_WOP + 8u * ks,
                   desc64(hi, lo_k + (ks * 2 * kGrp >> 4)), idk, 1u);
        }
        commit_one(one, done_kv);
        commit_one(one, kq_free + 8 * (it & 1));
        if (!kLocal) {
          wait_bar(rdy_p, it & 1, fail);
          wait_bar(done_kv, it & 1, fail);
          fence_after_sync();
#pragma unroll 1
          for (int ks = 0; ks < kC / 16; ++ks) {
            const uint32_t a = tm + T_VOP + 8u * ks;
            mma_ts(one, tm + T_PV, a, desc64(hi_p, lo_p + ((kstep(ks) + 8192) >> 4)), idn, ks > 0);
            if (kLo) mma_ts(one, tm + T_PV, a + 32u, desc64(hi_p, lo_p + (kstep(ks) >> 4)), idn, 1u);
          }
#pragma unroll 1
          for (int ks = 0; ks < kC / 16; ++ks)
            mma_ts(one, tm + T_PV, tm + T_VOP + 8u * ks,
                   desc64(hi_p, lo_p + (kstep(ks) >> 4)), idn, 1u);
          commit_one(one, done_o);
        }
      }
      commit_one(one, drain);  // arrives once every product issued above is done
      mbar_wait(drain, 0, kWaitLimit);
    }
    __syncwarp();
    cta_end();
    tmem_dealloc(tmem, 512);
  } else if (warp == kLoader) {
    // ===================================================== the copying warp
    int it = -1;
    for (Walk<kLocal> w(P); w.next();) {
      it = w.it;
      const uint32_t reg = sb + OFF_KQ + (it & 1) * kKQ, st = staged + 8 * (it & 1);
      // a unit's state on its way to L2 while the last chunk of the one before
      // is worked on
      if (!kLocal && w.first && lane == 0) {
        const size_t at = ((size_t)w.head * P.nseg + w.seg) * kD * kD;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                         (P.nseg > 1 ? P.ws_state : P.S) + at),
                     "r"((uint32_t)(kD * kD * sizeof(float)))
                     : "memory");
      }
      if (it >= 2) wait_bar(kq_free + 8 * (it & 1), ((it - 2) >> 1) & 1, fail);
      if (lane == 0) {
        mbar_expect(st, (kLocal ? 1u : 2u) * kC * kRow);
        tma_load(reg, &tm_k, w.vi / P.rep, w.c * kC, w.b, st);
        if (!kLocal) tma_load(reg + kC * kRow, &tm_q, w.vi / P.rep, w.c * kC, w.b, st);
      }
      __syncwarp();
      if (it >= 2) wait_bar(v_free + 8 * (it & 1), ((it - 2) >> 1) & 1, fail);
      if (lane == 0) {
        mbar_expect(vstaged + 8 * (it & 1), kC * kRow);
        tma_load(sb + OFF_V + (it & 1) * kV, &tm_v, w.vi, w.c * kC, w.b, vstaged + 8 * (it & 1));
      }
      __syncwarp();
    }
    // nothing may still be copying into shared memory when the CTA ends
    // (the last chunk of either parity)
    for (int j = max(it - 1, 0); j <= it; ++j) {
      mbar_wait(staged + 8 * (j & 1), (j >> 1) & 1, kWaitLimit);
      mbar_wait(vstaged + 8 * (j & 1), (j >> 1) & 1, kWaitLimit);
    }
    __syncwarp();
    cta_end();
  } else {
    // ====================================================== decay vectors
    // Two warps, chunk about (a chunk's vectors take one warp longer than the
    // other roles take for the chunk).  Lane l has tokens 2 l and 2 l + 1; log
    // decays to base 2.
    const int mine = warp - kGates;
    double total = 0.0;
    for (Walk<kLocal> w(P); w.next();) {
      const int it = w.it, nv = w.valid();
      if (w.first) total = 0.0;
      const bool store = kLocal && w.last() && lane == 0;
      double *sum = P.ws_decay + 2 * ((size_t)w.head * P.nseg + w.seg) + mine;
      if ((it & 1) != mine) {
        if (store) *sum = total;
        continue;
      }
      const size_t base = P.g_head ? (size_t)w.vi
                                   : ((size_t)w.b * P.T + (size_t)w.c * kC) * P.vh + w.vi;
      const size_t step = P.g_head ? 0 : (size_t)P.vh;
      Two G[2];  // cumulative
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        float x = t < nv ? __ldg(P.g + base + t * step) : 0.f;
        if (x < -1e4f) x = -1e4f;  // -inf: a decay that no float survives; NaN stays
        const float h = x * 1.44269502f;  // log2 e = 1.44269502 + 1.925963e-8
        G[i] = Two{h, fmaf(x, 1.44269502f, -h) + x * 1.925963033e-8f};
      }
      G[1] = add2(G[0], G[1]);
      Two run = G[1];
#pragma unroll 1
      for (int off = 1; off < 32; off <<= 1) {
        const Two y = shfl_up2(run, off);
        if (lane >= off) run = add2(run, y);
      }
      const Two end{__shfl_sync(0xffffffffu, run.h, 31), __shfl_sync(0xffffffffu, run.l, 31)};
      const Two before = shfl_up2(run, 1);
      if (lane > 0) {
        G[0] = add2(G[0], before);
        G[1] = add2(G[1], before);
      }
      total += (double)end.h + (double)end.l;
      float *vc = vec(it);
      // Gamma_t = gr + gf, and the decay from each token to the chunk's end,
      // 2^(dr + df): integer and rest, so that a weight has its bits however
      // small it is
      float gf[2], df[2];
      int gr[2], dr[2];
      auto parts = [](Two x, int &whole, float &rest) {
        const float r = rintf(x.h);
        whole = (int)r;
        rest = (x.h - r) + x.l;
      };
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        parts(G[i], gr[i], gf[i]);
        parts(add2(end, Two{-G[i].h, -G[i].l}), dr[i], df[i]);
      }
      int er;
      float ef;
      parts(end, er, ef);
      wait_bar(rdy_kq + 8 * (it & 1), (it >> 1) & 1, fail);
      const int *ex = rowexp(it);
      const int2 k2 = *reinterpret_cast<const int2 *>(ex + 2 * lane);
      const int kx[2] = {k2.x, k2.y};
      // (exactly; 0 below the normal floats, infinity above them)
      auto p2 = [](int e) { return e < -126 ? 0.f : pow2(min(e, 128)); };
      // The weight of row s in P[t], by its logarithm: r_s = -Gamma_s - kx_s,
      // and Gamma_t for every s.  R_t >= the largest r_s, s <= t, so P[t][s] =
      // G 2^{r_s - R_t - 22} keeps its bits whatever the decays and the rows'
      // sizes (|G| <= 2^37).
      float R[2] = {0.f, 0.f};
      bool some_row[2];  // some row up to this one is not zeros
      if (!kLocal) {
        const float none = -3e38f;
        float r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) r[i] = kx[i] < 127 ? -G[i].h - (float)kx[i] : none;
        float run_r = fmaxf(r[0], r[1]);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const float y = __shfl_up_sync(0xffffffffu, run_r, off);
          if (lane >= off) run_r = fmaxf(run_r, y);
        }
        const float before_r = __shfl_up_sync(0xffffffffu, run_r, 1);
        R[0] = ceilf(lane > 0 ? fmaxf(before_r, r[0]) : r[0]);
        R[1] = ceilf(run_r);
        // rows with nothing but zeros before them take the first other row's
        const unsigned some = __ballot_sync(0xffffffffu, R[1] > none);
        const float lo = some ? __shfl_sync(0xffffffffu, R[0] > none ? R[0] : R[1],
                                            __ffs(some) - 1)
                              : 0.f;
        const float hi = fmaxf(__shfl_sync(0xffffffffu, R[1], 31), lo);
        // one factor per row and column while their product cannot leave the
        // normal floats; otherwise an exponential per element
        const bool fac = hi - lo <= 120.f;
        const int c = -(int)rintf(0.5f * (hi + lo));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = 2 * lane + i;
          some_row[i] = R[i] > none;
          R[i] = fmaxf(R[i], lo);
          const int n = -22 - kx[i];
          vc[VA + t] = fac ? p2(-(int)R[i] - c) : -R[i];
          // (a key row of zeros: no weight, as R_t does not bound one)
          vc[VB + t] = kx[i] == 127 ? (fac ? 0.f : -1e30f)
                       : fac        ? ex2(-gf[i]) * p2(c + n - gr[i])
                                    : (float)n;
          vc[VGH + t] = G[i].h;
          vc[VGL + t] = G[i].l;
        }
        if (lane == 0) vc[VM + 1] = fac ? 1.f : 0.f;
      }
      // f_t = (decay to the end) / (k row scale), relative to a power of two
      // that bounds it: the largest of the rows that are finite and not zeros
      // (those have f = 0)
      bool row[2];
      int top = -1 << 24;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        row[i] = kx[i] > -114 && kx[i] < 127;
        if (row[i]) top = max(top, dr[i] - kx[i]);
      }
      const int fe = min(max(__reduce_max_sync(0xffffffffu, top) + 1, -126), 126);
      bool uneven = false;
      float f8 = 1.f;  // the least of the last 8 rows
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // (a k row that is not finite: the state is lost)
        const int t = 2 * lane + i;
        const float f = row[i]          ? ex2(df[i]) * p2(dr[i] - kx[i] - fe)
                        : kx[i] == 127 ? 0.f
                                       : __int_as_float(0x7fffffff);
        vc[VF + t] = f;
        uneven |= t < nv && f < 0x1p-17f;
        f8 = fminf(f8, f);
      }
      uneven = __any_sync(0xffffffffu, uneven);
      f8 = __uint_as_float(__reduce_min_sync(0xffffffffu, lane < 28 ? ~0u : __float_as_uint(f8)));
      if (lane == 0) {
        vc[VM] = ex2(ef) * p2(er);
        vc[VM + 2] = pow2(fe);
        vc[VM + 3] = uneven ? 0x1p17f * f8 : __int_as_float(0x7f800000);
      }
      if (!kLocal) {  // the output's factors
        const int2 q2 = *reinterpret_cast<const int2 *>(ex + 64 + 2 * lane);
        const int qx[2] = {q2.x, q2.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = 2 * lane + i;
          const float e = ex2(gf[i]);
          vc[VCA + t] = P.scale * (e * p2(gr[i] - qx[i] + kOutExp));
          // what P[t] and q_t are scaled by (where P[t] is all zeros, any)
          vc[VCB + t] =
              some_row[i] ? P.scale * (e * p2(gr[i] + (int)R[i] + 22 - qx[i] + kOutExp)) : 0.f;
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(vecs + 8 * (it & 3));
        if (store) *sum = total;
      }
    }
    if (kLocal) {  // segments without a chunk: no decay
      Walk<kLocal> w(P);
      for (int u = blockIdx.x; u < P.units; u += gridDim.x) {
        w.u = u;
        w.decode();
        if (w.c >= w.c_hi && lane == 0)
          P.ws_decay[2 * ((size_t)w.head * P.nseg + w.seg) + mine] = 0.0;
      }
    }
    cta_end();
  }
  }
}

// Start states of the segments from their own sums: for each head, in order,
// slot i takes the state before segment i and the state moves on by the
// segment's decay and sum.  One thread per two state elements; the sums of 32
// segments are asked for together and the decays worked out once a CTA (one
// after the other, in double precision in every thread, 18 segments of 8 heads
// took 20 us).
constexpr int kSegMax = 64;
__global__ void __launch_bounds__(256)
    linattn_chain_kernel(const float *__restrict__ S, float *__restrict__ ws,
                         const double *__restrict__ decay, int nseg) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kPer = kD * kD / 2;  // threads of a head, a multiple of a CTA's
  __shared__ float factor[kSegMax];
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t head = e / kPer, x = e % kPer;
  if ((int)threadIdx.x < nseg - 1) {
    const double *d2 = decay + 2 * (head * nseg + threadIdx.x), l = d2[0] + d2[1];
    const float h = (float)l, a = exp2f(h);
    factor[threadIdx.x] = fmaf(a, (float)(l - (double)h) * 0.69314718f, a);
  }
  float2 s = reinterpret_cast<const float2 *>(S)[e];
  float2 *w = reinterpret_cast<float2 *>(ws) + head * nseg * kPer + x;
  for (int i0 = 0; i0 < nseg; i0 += 32) {
    float2 d[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i0 + i < nseg - 1) d[i] = w[(size_t)(i0 + i) * kPer];
    if (i0 == 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i0 + i >= nseg) break;
      w[(size_t)(i0 + i) * kPer] = s;
      if (i0 + i < nseg - 1) {
        const float a = factor[i0 + i];
        s.x = fmaf(a, s.x, d[i].x);
        s.y = fmaf(a, s.y, d[i].y);
      }
    }
  }
}

// Segments per sequence.  One segment costs its chunks on the critical CTA;
// more segments run the KV pass too (half of the main pass per chunk, 0.6 with
// its launch)
// and read and write a start state each (about 2 chunks).  The cheapest
// count by that model.
int plan(int B, int vh, int T) {
  const long long heads = (long long)B * vh;
  const int n = (T + kC - 1) / kC;
  int best = 1;
  double cost = 1e300;
  for (int s = 1; s <= kSegMax && s <= n; ++s) {
    const long long waves = (heads * s + kSms - 1) / kSms;
    const double c = (double)waves * (((n + s - 1) / s) * (s > 1 ? 1.6 : 1.0) + (s > 1 ? 4 : 2));
    if (c < cost * 0.98) {
      cost = c;
      best = s;
    }
    if (heads * s >= 4LL * kSms) break;
  }
  return best;
}

// [B][T][heads][128] rows as a 4-d tensor {128, heads, T, B}; a box is 64
// token rows of one head.  Rows past T read as zeros.
cudaError_t rows_map(CUtensorMap *map, const void *base, bool bf16, int heads, int T, int B) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t row = (cuuint64_t)kD * (bf16 ? 2 : 4);
  const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t strides[3] = {row, row * (cuuint64_t)heads,
                                 row * (cuuint64_t)heads * (cuuint64_t)T};
  const cuuint32_t box[4] = {(cuuint32_t)kD, 1, (cuuint32_t)kC, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUresult r =
      fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
         const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Launched as a programmatic dependent of the kernel before it on the stream.
template <bool kBf16, bool kLocal>
cudaError_t launch(const CUtensorMap *m, const Args &a, cudaStream_t stream) {
  const auto kernel = linattn_chunk_kernel<kBf16, kLocal>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)min(a.units, kSms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], a);
}

}  // namespace

size_t linattn_prefill_workspace_bytes(int B, int vh, int T) {
  const size_t heads = (size_t)B * vh;
  const size_t nseg = (size_t)plan(B, vh, T);
  const size_t bytes = heads * nseg * (kD * kD * sizeof(float) + 2 * sizeof(double));
  return nseg == 1 ? 0 : (bytes + 15) & ~(size_t)15;
}

cudaError_t launch_linattn_prefill(const LinattnArgs &L, bool bf16, void *workspace,
                                   cudaStream_t stream) {
  const size_t heads = (size_t)L.B * L.vh;
  if (heads == 0) return cudaSuccess;
  const int nseg = plan(L.B, L.vh, L.M);
  if (heads * nseg > 0x7fffffffull / 256) return cudaErrorInvalidConfiguration;
  Args a;
  a.S = L.S_out;
  a.ws_state = static_cast<float *>(workspace);
  a.ws_decay = nseg > 1 ? reinterpret_cast<double *>(a.ws_state + heads * nseg * kD * kD) : nullptr;
  a.g = L.g;
  a.o = L.o;
  a.lens = L.lens;
  a.err = L.err;
  a.scale = L.scale;
  a.g_head = L.g_head;
  a.vh = L.vh;
  a.rep = L.rep;
  a.T = L.M;
  a.nseg = nseg;
  a.per_seg = ((L.M + kC - 1) / kC + nseg - 1) / nseg;
  CUtensorMap m[3];
  cudaError_t e;
  if ((e = rows_map(&m[0], L.q, bf16, L.kh, L.M, L.B)) != cudaSuccess) return e;
  if ((e = rows_map(&m[1], L.k, bf16, L.kh, L.M, L.B)) != cudaSuccess) return e;
  if ((e = rows_map(&m[2], L.v, bf16, L.vh, L.M, L.B)) != cudaSuccess) return e;
  if (nseg > 1) {
    a.units = (int)(heads * (nseg - 1));
    e = bf16 ? launch<true, true>(m, a, stream) : launch<false, true>(m, a, stream);
    if (e != cudaSuccess) return e;
    // (an ordinary launch: started early, all of it would land on the few SMs
    // that the pass before leaves free; 183 us for the one long prompt, not 145)
    linattn_chain_kernel<<<(unsigned)(heads * (kD * kD / 2 / 256)), 256, 0, stream>>>(
        a.S, a.ws_state, a.ws_decay, nseg);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  a.units = (int)(heads * nseg);
  return bf16 ? launch<true, false>(m, a, stream) : launch<false, false>(m, a, stream);
}

cudaError_t linattn_timeouts(unsigned int *count) {
  return cudaMemcpyFromSymbol(count, g_linattn_timeouts, sizeof(unsigned int));
}

}  // namespace gdn
