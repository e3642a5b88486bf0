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
// [-1, 1].  Error of an angle: 2^-53 pos of the frequency's own rounding plus 1e-7.
// A block makes the angles of its tokens once, in shared memory, for all of
// their heads.
//
// Borders between codes.  x / scale is divided to nearest and then made odd in
// its last bit where the division left a rest (the sign of the rest, exact by a
// fused multiply-add, says on which side), so that rounding it again to a code
// gives the code nearest to the true quotient.
//
// Layout.  8 channels a lane: 16 bytes of bf16 in and out, hd / 8 lanes a row,
// several rows a lane asked for at once.  Bound by HBM for prompts and by
// latency for single tokens.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "gdn_internal.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;  // tokens a block takes at most
constexpr int kRows = 4;        // rows a lane asks for at once

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

__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
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

// A row of 8 x kLanes values to its place in the cache.  Every lane of the warp
// takes part; `on`: this row is stored.
template <int kKind, int kLanes>
__device__ __forceinline__ void hold(const float (&x)[8], void *codes, float *scales, size_t row,
                                     int gl, bool on) {
  if (kKind == kKvBf16) {
    if (on) store8(static_cast<__nv_bfloat16 *>(codes) + row * (8 * kLanes) + 8 * gl, x);
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
  if (finite && scale > 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w.x |= code<kKind>(odd_quotient(x[i], scale)) << (8 * i);
      w.y |= code<kKind>(odd_quotient(x[4 + i], scale)) << (8 * i);
    }
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

// Turns and (kKind >= 0) the cache's rows.  A block takes P.tpc tokens and the
// heads [s0, s1) of q, k, v side by side that blockIdx.y has.
template <typename T, int kKind, int kLanes>
__global__ void __launch_bounds__(kThreads)
    kv_rows_kernel(const KvRows P) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kHd = 8 * kLanes, kGroups = kThreads / kLanes;
  __shared__ Token tokens[kMaxTokens];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, gl = tid % kLanes, group = tid / kLanes, lane = tid & 31;
  const long long tok0 = (long long)blockIdx.x * P.tpc;
  const int n = (int)min((long long)P.tpc, P.tokens - tok0);
  const int slots = P.qh + (kKind >= 0 ? 2 * P.c.kvh : 0);
  const int s0 = (int)blockIdx.y * P.spb, ns = min(P.spb, slots - s0), all = n * ns;
  const int half = P.half;
  unsigned long long *phase = reinterpret_cast<unsigned long long *>(smem);
  float2 *cs = reinterpret_cast<float2 *>(phase + half);

  auto source = [&](int r) -> const T * {
    const int t = r / ns, s = s0 + r - t * ns;
    const long long tok = tok0 + t;
    if (s < P.qh) return static_cast<const T *>(P.q) + tok * P.q_stride + s * kHd + 8 * gl;
    if (s < P.qh + P.c.kvh)
      return static_cast<const T *>(P.k) + tok * P.k_stride + (s - P.qh) * kHd + 8 * gl;
    return static_cast<const T *>(P.v) + tok * P.v_stride + (s - P.qh - P.c.kvh) * kHd + 8 * gl;
  };
  Raw<T> raw[kRows];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int j = 0; j < kRows; ++j)  // (rows past the end: the last one again)
      raw[j].load(source(min(r0 + j * kGroups + group, all - 1)));
  };
  fetch(0);

  if (tid < n) tokens[tid] = place(P, tok0 + tid);
  for (int i = tid; i < half; i += kThreads) {
    const double turns = P.freq[i] * 0.15915494309189533576888;  // 1 / 2 pi
    phase[i] = __double2ull_rd((turns - floor(turns)) * 18446744073709551616.0);
  }
  __syncthreads();
  for (int e = tid; e < n * half; e += kThreads) {
    const int t = e / half;
    const long long a = (long long)(phase[e - t * half] * (unsigned long long)(long long)tokens[t].pos);
    float s, c;
    sincospif(__ll2float_rn(a) * 1.0842021724855044e-19f, &s, &c);  // 2^-63
    cs[e] = make_float2(P.amp * c, P.amp * s);
  }
  __syncthreads();

  // the lane's place among the turned channels
  const int hl = half / 8;
  const bool pairs = P.pairs, upper = !pairs && gl >= hl;
  const bool turned = 8 * gl < 2 * half;
  const int f0 = pairs ? 4 * gl : 8 * (upper ? gl - hl : gl);
  const int other = lane - gl + (turned ? (upper ? gl - hl : gl + hl) : gl);
  for (int r0 = 0; r0 < all; r0 += kRows * kGroups) {
    Raw<T> now[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) now[j] = raw[j];
    if (r0 + kRows * kGroups < all) fetch(r0 + kRows * kGroups);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = r0 + j * kGroups + group;
      // (uniform over the warp: the rows of its first group come first)
      if (r0 + j * kGroups + (tid & ~31) / kLanes >= all) break;
      const int rc = min(r, all - 1), t = rc / ns, s = s0 + rc - t * ns;
      const Token &tk = tokens[t];
      const bool on = r < all && tk.on;
      float x[8];
      now[j].values(x);
      // v is not turned; whole warps skip the exchange where no row wants it
      const bool turn = half && s < P.qh + (kKind >= 0 ? P.c.kvh : 0);
      if (__any_sync(kFull, turn)) {
        const float2 *w = cs + t * half + f0;
        if (pairs) {
          if (turn && turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[2 * i], b = x[2 * i + 1];
              x[2 * i] = a * w[i].x - b * w[i].y;
              x[2 * i + 1] = b * w[i].x + a * w[i].y;
            }
          }
        } else {
          float y[8];
          now[j].partner(other, y);
          if (turn && turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * w[i].x + (upper ? y[i] : -y[i]) * w[i].y;
          }
        }
      }
      const long long tok = tok0 + t;
      if (s < P.qh && on)
        store8(static_cast<T *>(P.q_out) + (tok * P.qh + s) * kHd + 8 * gl, x);
      if (kKind >= 0) {
        const bool is_v = s >= P.qh + P.c.kvh, cached = s >= P.qh;
        if (__any_sync(kFull, cached)) {
          const int h = s - P.qh - (is_v ? P.c.kvh : 0);
          const size_t row = (size_t)tk.at + ((size_t)h << P.c.page_shift);
          hold<kKind < 0 ? 0 : kKind, kLanes>(x, is_v ? P.c.v : P.c.k, is_v ? P.c.v_scale : P.c.k_scale,
                                              row, gl, on && cached && tk.at >= 0);
        }
      }
    }
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = ((i < 4 ? a.x : a.y) >> (8 * (i & 3))) & 0xffu;
      if (kKind == kKvInt8) {
        x[i] = (float)(int)(signed char)c;
      } else {
        const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3);
        x[i] = __half2float(__half(h));
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

// Rows of the cache as k and v [B][M][kvh][hd].  A block takes P.tpc tokens.
template <typename T, int kKind, int kLanes>
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(const KvRows P) {
  constexpr int kHd = 8 * kLanes, kGroups = kThreads / kLanes;
  __shared__ Token tokens[kMaxTokens];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, gl = tid % kLanes, group = tid / kLanes;
  const long long tok0 = (long long)blockIdx.x * P.tpc;
  const int n = (int)min((long long)P.tpc, P.tokens - tok0);
  if (tid < n) tokens[tid] = place(P, tok0 + tid);
  __syncthreads();
  const int all = n * P.c.kvh;
  for (int r0 = group; r0 < all; r0 += kRows * kGroups) {
    Codes<kKind> k[kRows], v[kRows];
    float ks[kRows], vs[kRows];
    long long to[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = r0 + j * kGroups, t = r / P.c.kvh, h = r - t * P.c.kvh;
      to[j] = -1;
      if (r >= all || !tokens[t].on || tokens[t].at < 0) continue;
      const size_t row = (size_t)tokens[t].at + ((size_t)h << P.c.page_shift);
      to[j] = ((tok0 + t) * P.c.kvh + h) * kHd + 8 * gl;
      k[j].load(P.c.k, row * kHd + 8 * gl);
      v[j].load(P.c.v, row * kHd + 8 * gl);
      ks[j] = kKind == kKvBf16 ? 1.0f : __ldg(P.c.k_scale + row);
      vs[j] = kKind == kKvBf16 ? 1.0f : __ldg(P.c.v_scale + row);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (to[j] < 0) continue;
      float x[8];
      k[j].values(x);
      if (kKind != kKvBf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= ks[j];
      }
      store8(static_cast<T *>(P.q_out) + to[j], x);
      v[j].values(x);
      if (kKind != kKvBf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= vs[j];
      }
      store8(static_cast<T *>(P.v_out) + to[j], x);
    }
  }
}

template <typename T, int kKind, int kLanes>
cudaError_t rows_go(KvRows P, cudaStream_t stream, bool read) {
  const int heads = read ? P.c.kvh : P.qh + (kKind >= 0 ? 2 * P.c.kvh : 0);
  constexpr int kGroups = kThreads / kLanes;
  // Tokens of a block: as many as its groups' first rows cover, so that every
  // lane has kRows loads in flight.  Few tokens are cut by heads too: one
  // row a group then (64 tokens of 24 + 8 heads fill the GPU).
  constexpr int kFew = 152 * 4 * kGroups;  // rows that one row a group spreads over the SMs
  P.spb = heads;
  if (P.tokens * heads <= kFew) {
    P.tpc = kGroups / heads > 1 ? kGroups / heads : 1;
    if (!read && heads > kGroups) P.spb = kGroups;
  } else {
    P.tpc = kRows * kGroups / heads > 1 ? kRows * kGroups / heads : 1;
  }
  if (P.tpc > kMaxTokens) P.tpc = kMaxTokens;
  const long long blocks = (P.tokens + P.tpc - 1) / P.tpc;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)((heads + P.spb - 1) / P.spb));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = read ? 0 : (size_t)P.half * 8 * (1 + P.tpc);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (kKind >= 0) {
    if (read) return cudaLaunchKernelEx(&cfg, kv_read_kernel<T, kKind, kLanes>, P);
  }
  const auto kernel = kv_rows_kernel<T, kKind, kLanes>;
  if (cfg.dynamicSmemBytes > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, kernel, P);
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
