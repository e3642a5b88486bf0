// Rotary positions, writing a paged key-value cache, and reading it back, for
// sm_103a (gdn_rope_m, gdn_kv_write_m, gdn_kv_read).
//
// What they compute.  A row is one head of one token, hd channels.
//   turn   pair i of the first rot channels by the angle pos freq[i]:
//          (x, y) -> amp (x cos - y sin, y cos + x sin)
//   hold   bf16: rounded once.  8 bits: scale = max|row| / 127 (448 for e4m3),
//          code = the nearest of x / scale, ties to even
//   read   code scale
//
// Angles.  fp32 products of positions and frequencies are off by whole radians
// at far positions (2^20 x 2^-24), so a frequency is held as turns a position
// in 64-bit fixed point: pos times it is exact modulo one turn, an integer
// product drops the whole turns, and the rest goes to sincospif as a number in
// [-1, 1], with what its rounding to a float left of it added to first order.
// Error of an angle: 2^-64 pos turns, of the frequency as it is given.
// hd / 8 lanes take a token and a run of its heads, and keep its cosines and sines
// in registers.
//
// Borders between codes.  x (1 / scale) is within 2^-22 of the quotient, which
// settles the code but where a border lies that near; there x / scale is divided
// to nearest and made odd in its last bit where the division left a rest (the sign
// of the rest, exact by a fused multiply-add, says on which side), so that
// rounding it again gives the code nearest to the true quotient.
//
// Layout.  8 channels a lane: 16 bytes of bf16 in and out, hd / 8 lanes a row,
// several rows a lane asked for at once.
//
// Measured: 32768 rows x 32 heads of 128, bf16, whole heads turned: 88 us (537 MB,
// 90 % of the copy rate).  8 prompts of 4096 tokens x 32 + 16 heads into bf16 136 us
// (all of the copy rate), into e4m3 144 us (89 %: the rounding of k and v, 40 % of the
// instructions, beside the loads); padded ones of up to 4096 tokens 79 and 71 us, and
// back from e4m3 18 us.  65531 positions x 4 heads of 256, int8 to bf16: 65 us (91 %);
// 8 x 65531 positions of 128 channels, int8 to bf16: 1 head 76 % of the copy rate, 2
// heads 69, 3 83, 4 92.  64 tokens of 24 + 8 heads: 4.0 us a kernel, the chain from
// lengths to pages and rows to stores.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "gdn_internal.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kMaxHalf = 128;  // pairs of a head

// What a block knows of a token.
struct Token {
  long long at;  // page * kvh * page rows + row in the page, or -1: no place
  int pos;
  int on;
};

// 8 elements as they lie in memory (by plain loads: rows may be turned in place).
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  // (the other lane's)
  __device__ __forceinline__ void partner(int lane, float (&x)[8]) const {
    values(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __shfl_sync(kFull, x[i], lane);
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    a = *reinterpret_cast<const uint4 *>(p);
  }
  static __device__ __forceinline__ void wide(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const { wide(a, x); }
  __device__ __forceinline__ void partner(int lane, float (&x)[8]) const {
    uint4 u;
    u.x = __shfl_sync(kFull, a.x, lane);
    u.y = __shfl_sync(kFull, a.y, lane);
    u.z = __shfl_sync(kFull, a.z, lane);
    u.w = __shfl_sync(kFull, a.w, lane);
    wide(u, x);
  }
};

__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 elements of a row to p; `group`: the row's lanes, all of which store.  fp32:
// neighbours exchange halves, so that a store fills whole sectors.
__device__ __forceinline__ void store8(float *p, const float (&x)[8], unsigned group) {
  const bool odd = threadIdx.x & 1;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __shfl_xor_sync(group, odd ? x[i] : x[4 + i], 1);
  float4 *to = reinterpret_cast<float4 *>(p) - (odd ? 1 : 0);
  to[0] = odd ? make_float4(y[0], y[1], y[2], y[3]) : make_float4(x[0], x[1], x[2], x[3]);
  to[2] = odd ? make_float4(x[4], x[5], x[6], x[7]) : make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8], unsigned) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(two_bf16(x[0], x[1]), two_bf16(x[2], x[3]),
                                             two_bf16(x[4], x[5]), two_bf16(x[6], x[7]));
}

// x / s, the last bit set where the quotient is not exact (s a positive number).
__device__ __forceinline__ float odd_quotient(float x, float s) {
  const float q = __fdiv_rn(x, s);
  const float r = __fmaf_rn(-q, s, x);
  int b = __float_as_int(q);
  if (r != 0.0f) b = (b - ((r < 0.0f) != (x < 0.0f) ? 1 : 0)) | 1;
  return __int_as_float(b);
}

template <int kKind>
__device__ __forceinline__ uint32_t code(float q) {
  if (kKind == kKvInt8)
    return (uint32_t)(__float2int_rn(fminf(fmaxf(q, -127.0f), 127.0f))) & 0xffu;
  return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

// The codes nearest to x / s in place of the bytes of w that `which` has bits of.
template <int kKind>
__device__ __forceinline__ uint32_t settle(uint32_t w, uint32_t which, const float *x, float s) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (which >> (8 * i) & 0xffu)
      w = (w & ~(0xffu << (8 * i))) | code<kKind>(odd_quotient(x[i], s)) << (8 * i);
  return w;
}

// The codes of four elements of a row with scale s.
template <int kKind>
__device__ __forceinline__ uint32_t codes4(const float *x, float s, float inv) {
  uint32_t w;
  if (kKind == kKvInt8) {
    // rounded by the addition of 1.5 2^23; what that took off says how near the
    // border is (the quotient is within 127 2^-22 of x inv)
    constexpr float kBig = 12582912.0f;
    uint32_t u[4];
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float q = x[i] * inv, t = q + kBig;
      u[i] = __float_as_uint(t);
      far = fmaxf(far, fabsf(q - (t - kBig)));
    }
    w = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    if (far > 0.4999f) w = settle<kKind>(w, ~0u, x, s);
  } else {
    // the codes of both ends of where the quotient may lie
    const float up = inv * (1.0f + 0x1p-21f), dn = inv * (1.0f - 0x1p-21f);
    uint32_t a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * dn, x[2 * i + 1] * dn), __NV_SATFINITE,
                                      __NV_E4M3);
      b[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * up, x[2 * i + 1] * up), __NV_SATFINITE,
                                      __NV_E4M3);
    }
    w = a[0] | a[1] << 16;
    const uint32_t d = w ^ (b[0] | b[1] << 16);
    if (d) w = settle<kKind>(w, d, x, s);
  }
  return w;
}

// A row of 8 x kLanes values to its place in the cache.  Every lane of the warp
// takes part; `on`: this row is stored.
template <int kKind, int kLanes>
__device__ __forceinline__ void hold(const float (&x)[8], void *codes, float *scales, size_t row,
                                     int gl, bool on) {
  if (kKind == kKvBf16) {
    if (on) store8(static_cast<__nv_bfloat16 *>(codes) + row * (8 * kLanes) + 8 * gl, x, 0u);
    return;
  }
  // the largest as bits: infinities and NaN are above every number
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int d = 1; d < kLanes; d *= 2) top = max(top, __shfl_xor_sync(kFull, top, d));
  if (!on) return;
  const bool finite = top < 0x7f800000u;
  const float scale = finite ? __fdiv_rn(__uint_as_float(top), kKind == kKvInt8 ? 127.0f : 448.0f)
                             : __uint_as_float(0x7fc00000u);
  uint2 w = make_uint2(0, 0);
  if (finite && scale >= 0x1p-100f) {
    const float inv = __frcp_rn(scale);
    w.x = codes4<kKind>(x, scale, inv);
    w.y = codes4<kKind>(x + 4, scale, inv);
  } else if (finite && scale > 0.0f) {  // (its reciprocal or the rests would not be exact enough)
    w.x = settle<kKind>(0u, ~0u, x, scale);
    w.y = settle<kKind>(0u, ~0u, x + 4, scale);
  }
  *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(codes) + row * (8 * kLanes) + 8 * gl) = w;
  if (gl == 0) scales[row] = scale;
}

// Where the tokens of a block go (positions given: rope alone).
__device__ __forceinline__ Token place(const KvRows &P, long long tok) {
  Token t{-1, 0, 1};
  if (P.pos) {
    t.pos = P.pos[tok];
    return t;
  }
  const int b = (int)(tok / P.M), m = (int)(tok - (long long)b * P.M);
  const int start = P.start ? P.start[b] : 0, n = P.counts ? P.counts[b] : P.M;
  const long long room = (long long)P.cols << P.c.page_shift;
  if (n == 0) {  // left out, whatever its start
    t.on = 0;
    return t;
  }
  if (n < 0 || n > P.M || start < 0 || (long long)start + n > room) {
    t.on = 0;
    if (m == 0 && P.err) *P.err = 1;
    return t;
  }
  t.on = m < n;
  if (!t.on) return t;
  t.pos = start + m;
  const int page = P.table[(size_t)b * P.cols + (t.pos >> P.c.page_shift)];
  if ((unsigned)page < (unsigned)P.c.pages)
    t.at = (((long long)page * P.c.kvh) << P.c.page_shift) + (t.pos & ((1 << P.c.page_shift) - 1));
  else if (P.err)
    *P.err = 1;
  return t;
}

// The lanes of a row, of kLanes.
template <int kLanes>
__device__ __forceinline__ unsigned lanes_of_row() {
  return kLanes == 32 ? kFull : ((1u << (kLanes & 31)) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
}

// Turns and (kKind >= 0) the cache's rows.  A warp takes 32 / kLanes tokens, each
// with kLanes lanes, and a run of P.run of their heads (q, k and v side by side),
// the same for all warps of a block: blocks with rows to round and blocks without
// end apart.
template <typename T, int kKind, int kLanes>
__global__ void __launch_bounds__(kThreads, 4)
    kv_rows_kernel(const KvRows P) {
  constexpr int kHd = 8 * kLanes, kTokens = 32 / kLanes;
  __shared__ unsigned long long phase[kMaxHalf];
  __shared__ float amps[kMaxHalf];  // NaN for a frequency that is not finite
  __shared__ float2 angles[4 * kThreads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, gl = tid % kLanes, lane = tid & 31, half = P.half;
  const unsigned group = lanes_of_row<kLanes>();
  const int turned_heads = P.qh + (kKind >= 0 ? P.c.kvh : 0);
  const int slots = turned_heads + (kKind >= 0 ? P.c.kvh : 0);
  const int runs = (slots + P.run - 1) / P.run;
  const long long first = ((long long)(blockIdx.x / runs) * (kThreads / 32) + (tid >> 5)) * kTokens;
  const int s0 = (int)(blockIdx.x % runs) * P.run, s1 = min(s0 + P.run, slots);
  const bool there = first + lane / kLanes < P.tokens;
  // (past the end: the last token again, storing nothing)
  const long long tok = there ? first + lane / kLanes : P.tokens - 1;

  auto fetch = [&](Raw<T> &raw, int x) {
    const T *p = x < P.qh ? static_cast<const T *>(P.q) + tok * P.q_stride + x * kHd
                 : x < turned_heads
                     ? static_cast<const T *>(P.k) + tok * P.k_stride + (x - P.qh) * kHd
                     : static_cast<const T *>(P.v) + tok * P.v_stride + (x - turned_heads) * kHd;
    raw.load(p + 8 * gl);
  };
  // One row a lane: it is asked for beside the lengths and pages.  Longer runs
  // ask behind them, so that rows of padding are left where they are (8 padded
  // prompts of 4096 tokens: half of the bytes).
  const bool single = P.run == 1;
  Raw<T> one;
  if (single) fetch(one, s0);
  const Token tk = place(P, tok);
  const bool on = there && tk.on;

  // the lane's place among the turned channels, and its angles
  const bool pairs = P.pairs, upper = !pairs && 8 * gl >= half;
  const bool turned = 8 * gl < 2 * half;
  const int other = lane + (turned && !pairs ? (upper ? -(half / 8) : half / 8) : 0);
  float c[8], w[8];  // (pairs side by side: the first four)
  if (half) {
    for (int i = tid; i < half; i += kThreads) {
      // of |freq|, negated after it: turning back is the mirror image to the bit
      constexpr double kTurn = 0.15915494309189533577, kRest = -9.839338337591243e-18;  // 1 / 2 pi
      const double f = P.freq[i], a = fabs(f), turns = a * kTurn;
      // (and what the product and the constant's rounding left of it)
      const double rest = fma(a, kTurn, -turns) + a * kRest;
      const unsigned long long p = __double2ull_rd((turns - floor(turns)) * 0x1p64) +
                                   (unsigned long long)__double2ll_rn(rest * 0x1p64);
      phase[i] = f < 0.0 ? 0ull - p : p;
      amps[i] = a < INFINITY ? P.amp : __uint_as_float(0x7fc00000u);
    }
    __syncthreads();
  }
  if (!__any_sync(kFull, on)) return;
  if (half && s0 < turned_heads) {
    // the token's angles, each by one of its lanes
    float2 *const cs = angles + (tid / kLanes) * (4 * kLanes);
#pragma unroll 1
    for (int i = gl; i < half; i += kLanes) {
      const long long a = (long long)(phase[i] * (unsigned long long)(long long)tk.pos);
      // the angle as a float and what its rounding left of it, to first order
      const float near = __ll2float_rn(a);
      const float rest = __ll2float_rn(a - __float2ll_rn(near)) * 3.4061215800865545e-19f;  // pi 2^-63
      float x, y;
      sincospif(near * 1.0842021724855044e-19f, &y, &x);  // 2^-63
      cs[i] = make_float2(amps[i] * (x - y * rest), amps[i] * (y + x * rest));
    }
    __syncwarp();
    const int f0 = !turned ? 0 : pairs ? 4 * gl : 8 * gl - (upper ? half : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = cs[pairs ? f0 + (i & 3) : f0 + i];
      c[i] = x.x;
      w[i] = upper || pairs ? x.y : -x.y;  // (of the partner)
    }
  }
  // (every lane of the warp is at the same head)
  auto turn = [&](const Raw<T> &raw, float (&y)[8]) {
    if (pairs) {
      if (!turned) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = a * c[i] - b * w[i];
        y[2 * i + 1] = b * c[i] + a * w[i];
      }
    } else {
      float z[8];
      raw.partner(other, z);
      if (!turned) return;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * c[i] + z[i] * w[i];
    }
  };
  auto row_q = [&](const Raw<T> &raw, int x) {
    float y[8];
    raw.values(y);
    if (half) turn(raw, y);
    if (on) store8(static_cast<T *>(P.q_out) + (tok * P.qh + x) * kHd + 8 * gl, y, group);
  };
  auto row_kv = [&](const Raw<T> &raw, int x) {
    if constexpr (kKind >= 0) {
      float y[8];
      raw.values(y);
      if (half && x < turned_heads) turn(raw, y);
      const bool is_v = x >= turned_heads;
      const int h = x - (is_v ? turned_heads : P.qh);
      hold<kKind, kLanes>(y, is_v ? P.c.v : P.c.k, is_v ? P.c.v_scale : P.c.k_scale,
                          (size_t)tk.at + ((size_t)h << P.c.page_shift), gl, on && tk.at >= 0);
    }
  };
  if (single) {
    if (s0 < P.qh)
      row_q(one, s0);
    else
      row_kv(one, s0);
    return;
  }
  constexpr int kQ = sizeof(T) == 2 ? 4 : 2, kKv = 2;  // rows under way
  const int q1 = min(s1, P.qh);
#pragma unroll 1
  for (int x = s0; x < q1; x += kQ) {
    Raw<T> raw[kQ];
#pragma unroll
    for (int j = 0; j < kQ; ++j) fetch(raw[j], min(x + j, q1 - 1));
#pragma unroll
    for (int j = 0; j < kQ; ++j)
      if (x + j < q1) row_q(raw[j], x + j);
  }
  const int k0 = max(s0, P.qh);
  Raw<T> next[kKv];
  if (k0 < s1) {
#pragma unroll
    for (int j = 0; j < kKv; ++j) fetch(next[j], min(k0 + j, s1 - 1));
  }
#pragma unroll 1
  for (int x = k0; x < s1; x += kKv) {
    Raw<T> raw[kKv];
#pragma unroll
    for (int j = 0; j < kKv; ++j) {
      raw[j] = next[j];
      fetch(next[j], min(x + kKv + j, s1 - 1));
    }
#pragma unroll
    for (int j = 0; j < kKv; ++j)
      if (x + j < s1) row_kv(raw[j], x + j);
  }
}

// 8 codes of a row as numbers.
template <int kKind>
struct Codes {
  uint2 a;
  __device__ __forceinline__ void load(const void *p, size_t at) {
    a = __ldg(reinterpret_cast<const uint2 *>(static_cast<const unsigned char *>(p) + at));
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if (kKind == kKvInt8) {  // code + 128 behind the bits of 2^23
      const uint32_t w[2] = {a.x ^ 0x80808080u, a.y ^ 0x80808080u};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = __uint_as_float(__byte_perm(w[i / 4], 0x4b000000u, 0x7540 + (i & 3))) - 8388736.0f;
    } else {
      const uint32_t w[4] = {a.x, a.x >> 16, a.y, a.y >> 16};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(
            __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] & 0xffffu), __NV_E4M3)));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};
template <>
struct Codes<kKvBf16> {
  Raw<__nv_bfloat16> r;
  __device__ __forceinline__ void load(const void *p, size_t at) {
    r.load(static_cast<const __nv_bfloat16 *>(p) + at);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const { r.values(x); }
};

// Rows of the cache as k and v [B][M][kvh][hd]: kLanes lanes take a token and
// P.run of its heads, K and V of four at a time; of a single head (kOne) the rows
// of four tokens, so that as much is under way.
template <typename T, int kKind, int kLanes, bool kOne>
__global__ void __launch_bounds__(kThreads, 4)
    kv_read_kernel(const KvRows P) {
  constexpr int kHd = 8 * kLanes, kGroups = kThreads / kLanes;
  constexpr int kRows = 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, gl = tid % kLanes, kvh = P.c.kvh;
  const unsigned group = lanes_of_row<kLanes>();
  const long long job = (long long)blockIdx.x * kGroups + tid / kLanes;
  const int runs = (kvh + P.run - 1) / P.run;
  const long long tok = kOne ? job * kRows : job / runs;
  if (tok >= P.tokens) return;
  const int h0 = kOne ? 0 : (int)(job - tok * runs) * P.run, h1 = kOne ? kRows : min(h0 + P.run, kvh);
  Token tk[kOne ? kRows : 1];
#pragma unroll
  for (int i = 0; i < (kOne ? kRows : 1); ++i) {
    tk[i] = Token{-1, 0, 0};
    if (tok + i < P.tokens) tk[i] = place(P, tok + i);
  }
  if (!kOne && (!tk[0].on || tk[0].at < 0)) return;
#pragma unroll 1
  for (int h = h0; h < h1; h += kRows) {
    Codes<kKind> k[kRows], v[kRows];
    float ks[kRows], vs[kRows];
    bool there[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const Token &t = tk[kOne ? j : 0];
      there[j] = kOne ? t.on && t.at >= 0 : h + j < h1;
      if (!there[j]) continue;
      const size_t row = (size_t)t.at + ((size_t)(kOne ? 0 : h + j) << P.c.page_shift);
      k[j].load(P.c.k, row * kHd + 8 * gl);
      v[j].load(P.c.v, row * kHd + 8 * gl);
      ks[j] = kKind == kKvBf16 ? 1.0f : __ldg(P.c.k_scale + row);
      vs[j] = kKind == kKvBf16 ? 1.0f : __ldg(P.c.v_scale + row);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (!there[j]) continue;
      const long long to = (tok * kvh + h + j) * kHd + 8 * gl;  // (kOne: of token tok + j)
      float x[8];
      k[j].values(x);
      if (kKind != kKvBf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= ks[j];
      }
      store8(static_cast<T *>(P.q_out) + to, x, group);
      v[j].values(x);
      if (kKind != kKvBf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= vs[j];
      }
      store8(static_cast<T *>(P.v_out) + to, x, group);
    }
  }
}

template <typename T, int kKind, int kLanes>
cudaError_t rows_go(KvRows P, cudaStream_t stream, bool read) {
  const int heads = read ? P.c.kvh : P.qh + (kKind >= 0 ? 2 * P.c.kvh : 0);
  constexpr int kGroups = kThreads / kLanes;
  // A run is as long as leaves four blocks for every SM, in steps of the rows
  // under way: single tokens are cut down to a row a group (64 tokens of
  // 24 + 8 heads fill the GPU), prompts take all of a token's heads for one
  // set of angles.
  const long long rows = P.tokens * heads, full = 152ll * 4 * kGroups;
  const int step = read || sizeof(T) == 2 ? 4 : 2;
  long long run = (rows + full - 1) / full;
  if (run > 1) run = (run + step - 1) / step * step;
  P.run = (int)(run < heads ? run : heads);
  const long long runs = (heads + P.run - 1) / P.run;
  constexpr int kTokens = 32 / kLanes;
  // Four tokens a job pay from 24000 rows on, whatever they hold: with one and
  // with four, 20000 rows 5.3 and 4.9 us (128 channels, int8 to bf16), 3.5 and 3.8
  // (64, bf16), 12.2 and 13.2 (256, e4m3 to fp32); 30000 rows 7.0 and 6.5, 4.1 and 4.0,
  // 17.5 and 17.0; 1.8 million rows 402 and 261, 219 and 136, 905 and 746.
  const bool one = read && heads == 1 && rows > 24000;
  const long long jobs = one ? (P.tokens + 3) / 4 : P.tokens * runs;
  const long long blocks = read ? (jobs + kGroups - 1) / kGroups
                                : (P.tokens + 8 * kTokens - 1) / (8 * kTokens) * runs;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (kKind >= 0) {
    if (read)
      return one ? cudaLaunchKernelEx(&cfg, kv_read_kernel<T, kKind, kLanes, true>, P)
                 : cudaLaunchKernelEx(&cfg, kv_read_kernel<T, kKind, kLanes, false>, P);
  }
  return cudaLaunchKernelEx(&cfg, kv_rows_kernel<T, kKind, kLanes>, P);
}

template <typename T, int kKind>
cudaError_t by_head(const KvRows &P, int hd, cudaStream_t stream, bool read) {
  return hd == 64    ? rows_go<T, kKind, 8>(P, stream, read)
         : hd == 128 ? rows_go<T, kKind, 16>(P, stream, read)
                     : rows_go<T, kKind, 32>(P, stream, read);
}

template <typename T>
cudaError_t by_kind(const KvRows &P, int hd, cudaStream_t stream, bool read) {
  if (P.pos) return by_head<T, -1>(P, hd, stream, false);
  return P.c.kind == kKvBf16   ? by_head<T, kKvBf16>(P, hd, stream, read)
         : P.c.kind == kKvInt8 ? by_head<T, kKvInt8>(P, hd, stream, read)
                               : by_head<T, kKvE4m3>(P, hd, stream, read);
}

}  // namespace

cudaError_t launch_kv_rows(const KvRows &P, int hd, bool bf16, bool read, cudaStream_t stream) {
  if (P.tokens == 0) return cudaSuccess;
  return bf16 ? by_kind<__nv_bfloat16>(P, hd, stream, read) : by_kind<float>(P, hd, stream, read);
}

}  // namespace gdn
