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
// bits).  With bf16 rows q, k and v fit one fp16 each; the scores and the
// state that enter o are rounded to fp16 (2^-11, below o's own 2^-8), and the
// decayed values that enter the state stay hi + lo.  The scales: q and k by
// row, v, the decayed values and the state by column dv (the TMEM lane),
// chosen so that the largest element lies in [2^14, 2^15); elements down to
// 2^-17 of it keep all their bits.  The scores of row t are scaled by the
// largest k row up to t.  The state is kept in fp32 registers: a chunk's KV
// product is read out, unscaled and added, so scales may differ from chunk to
// chunk.  Gamma is summed in fp64 and its differences are split into two
// floats, so strong decays keep the small differences between near tokens.
//
// Roles (20 warps, one CTA per SM, persistent over (sequence, head, segment)
// units): 8 warps A hold the state and make its operand and the two V
// operands; 8 warps B turn the staged q and k rows into operands in place,
// make P from G, and the output from QS and PV; one warp issues the products,
// one copies rows by TMA (a chunk ahead), one computes the decay vectors.
// All meet through mbarriers; the chunks of successive units form one
// sequence, so a unit's first loads run under the previous one's last chunk.
//
// Few heads: a sequence is cut into segments (see plan()); a first pass
// of the same kernel computes each segment's own contribution to the state
// (KV only), a second kernel chains them into every segment's start state, and
// the main pass runs over all segments at once.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "gdn_internal.cuh"
#include "gdn_tc.cuh"

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
// chunk's staged rows (K then Q), converted in place to the [K; Q] operand:
// 128 rows x 128 fp16, 128-byte swizzle, the hi tile then the lo tile.
constexpr uint32_t OFF_KQ = 0, kKQ = 65536;   // by chunk parity
constexpr uint32_t OFF_V = 131072;            // staged v rows [64][128]
constexpr uint32_t OFF_O = 163840;            // o tile [64][128]
constexpr uint32_t OFF_P = 196608;            // P operand 64 x 64, hi, lo
// decay vectors of a chunk, buffer it & 3, 512 floats:
constexpr int VA = 0, VB = 64, VF = 128, VCA = 192, VCB = 256, VGH = 320,
              VGL = 384, VM = 448;
constexpr uint32_t OFF_VEC = 212992;
constexpr uint32_t OFF_EXP = OFF_VEC + 4 * 2048;    // row exponents [2][128]
constexpr uint32_t OFF_LANE = OFF_EXP + 2 * 512;    // lane factors [4][2][128]
constexpr uint32_t OFF_PV = OFF_LANE + 4 * 1024;    // exchange: V maxima
constexpr uint32_t OFF_PS = OFF_PV + 2048;          // exchange: state maxima
constexpr uint32_t OFF_BAD = OFF_PS + 1024;         // first bad token [4][2][128]
constexpr uint32_t OFF_BAR = OFF_BAD + 1024;
constexpr uint32_t kSmemUsed = OFF_BAR + 256;
constexpr uint32_t kSmemAlloc = kSmemUsed + 1024;   // room to align the base
static_assert(kSmemAlloc <= 232448, "shared memory");

// TMEM columns (512): the KV product, the state operand (hi, lo), the V and
// decayed V operands (hi, lo), QS, and G, which PV overwrites once P is made.
constexpr uint32_t T_D = 0, T_SOP = 128, T_VOP = 256, T_WOP = 320, T_QS = 384,
                   T_G = 448;

__host__ __device__ constexpr uint32_t idesc16(int M, int N, int b_mn) {
  // fp16 operands (format 0), fp32 accumulator; B MN-major if b_mn
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

struct Args {
  float *S;             // [B][vh][128][128], in/out
  float *ws_state;      // [B vh][nseg][128][128]: own sums, then start states
  double *ws_decay;     // [B vh][nseg]: log2 of a segment's decay
  const float *g;
  void *o;
  const int *lens;
  int *err;
  float scale;
  int g_head, vh, rep, T, nseg, nchunks, units;
};

// ------------------------------------------------------------- sequencing

// The chunks this CTA works on, in order; every role walks the same list.
template <bool kLocal>
struct Walk {
  const Args *p;
  int u, c, c_hi, it;   // unit, chunk, end of its chunks, running index
  int head, b, vi, seg, n;
  bool ok, first;
  __device__ Walk(const Args &P) : p(&P), u((int)blockIdx.x - (int)gridDim.x), it(0) {
    unit();
  }
  // Decodes unit u; false if its sequence has no valid length.
  __device__ bool decode() {
    const int per = kLocal ? p->nseg - 1 : p->nseg;
    head = u / per;
    seg = u - head * per;
    b = head / p->vh;
    vi = head - b * p->vh;
    n = p->lens ? __ldg(p->lens + b) : p->T;
    const bool good = n >= 0 && n <= p->T;
    if (!good) n = 0;
    c = (int)((long long)seg * p->nchunks / p->nseg);
    c_hi = min((int)((long long)(seg + 1) * p->nchunks / p->nseg), (n + kC - 1) / kC);
    return good;
  }
  __device__ void unit() {
    first = true;
    for (;;) {
      u += gridDim.x;
      ok = u < p->units;
      if (!ok) return;
      decode();
      if (c < c_hi) return;
    }
  }
  __device__ void next() {
    ++it;
    first = false;
    if (++c >= c_hi) unit();
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

// max |x| that keeps NaN (as a bit pattern above infinity's)
__device__ __forceinline__ float amax(float m, float x) {
  return __int_as_float(max(__float_as_int(m), __float_as_int(x) & 0x7fffffff));
}

__device__ __forceinline__ uint32_t h2_bits(__half2 v) {
  return *reinterpret_cast<uint32_t *>(&v);
}

template <bool kLo>
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(a, b);
  hi = h2_bits(h);
  if (kLo) {
    const float2 f = __half22float2(h);
    lo = h2_bits(__floats2half2_rn(a - f.x, b - f.y));
  }
}

// Columns c0 .. c0+7 of row r of an R x C tile (hi; lo behind it), times s.
template <bool kLo>
__device__ __forceinline__ void put8(unsigned char *gb, uint32_t off, int R, int C,
                                     int r, int c0, const float *x, float s) {
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2<kLo>(x[2 * i] * s, x[2 * i + 1] * s, hi[i], lo[i]);
  const uint32_t o = off + sw128_off(R, r, c0, 2);
  *reinterpret_cast<uint4 *>(gb + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  if (kLo)
    *reinterpret_cast<uint4 *>(gb + o + (uint32_t)(R * C * 2)) =
        make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// Elements c0 .. c0+15 of this lane of an A operand in TMEM, times s.
template <bool kLo>
__device__ __forceinline__ void put16(uint32_t hi, uint32_t lo, int c0,
                                      const float *x, float s) {
  uint32_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split2<kLo>(x[2 * i] * s, x[2 * i + 1] * s, h[i], l[i]);
  tmem_st8_async(hi + (uint32_t)(c0 >> 1), h);
  if (kLo) tmem_st8_async(lo + (uint32_t)(c0 >> 1), l);
}

// 32 TMEM columns of this thread's lane; tmem_wait_ld before use.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&u)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]),
        "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]),
        "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]),
        "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]),
        "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}

template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&u)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // the loaded registers are defined only from here on
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(u[i]));
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
  for (uint32_t i = 0; i < kWaitLimit; i += 256) {
    if (mbar_wait(bar, parity, 256)) return;
    if (*fail) return;
  }
  *fail = 1;
}

__device__ __forceinline__ void signal_ready(uint32_t mbar) {
  fence_proxy_async();
  fence_before_sync();
  mbar_arrive(mbar);
}

__device__ __forceinline__ void bar_pair(int quad) {  // warps w and w + 4 of A
  asm volatile("bar.sync %0, 64;" ::"r"(quad + 1) : "memory");
}

__device__ __forceinline__ void bar_b() {
  asm volatile("bar.sync 5, %0;" ::"n"(kGroup) : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t smem, const CUtensorMap *map, int h,
                                         int t0, int b, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(h), "r"(t0), "r"(b), "r"(mbar)
      : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap *map, int h, int t0, int b,
                                          uint32_t smem) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group"
      " [%0, {%1, %2, %3, %4}], [%5];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(0), "r"(h), "r"(t0), "r"(b), "r"(smem)
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// ---------------------------------------------------------------- products

// Shared-memory operand tile of R rows, C columns: descriptor of K step ks of
// the hi (part 0) or lo tile.  K-major: rows are M or N.  MN-major: rows are K.
__device__ __forceinline__ uint64_t kdesc(uint32_t base, int R, int ks) {
  return desc_kstep(base, R, ks);
}

__device__ __forceinline__ uint64_t mndesc(uint32_t base, int R, int ks) {
  uint64_t d = desc_sw128(base + (uint32_t)ks * 2048u);
  d &= ~((uint64_t)0x3FFF << 16);
  d |= (uint64_t)(((uint32_t)R * 128u) >> 4) << 16;
  return d;
}

// ------------------------------------------------------------------ kernel

template <bool kBf16, bool kLocal>
__global__ void __launch_bounds__(kThreads, 1)
    linattn_chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ CUtensorMap tm_o,
                         const __grid_constant__ Args P) {
  constexpr bool kLo = !kBf16;                 // second parts of q, k, v, P, S
  constexpr uint32_t kRow = kBf16 ? 256 : 512; // bytes of a token row
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_s = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t sb = (raw_s + 1023u) & ~1023u;
  unsigned char *gb = smem_raw + (sb - raw_s);
  const uint32_t bar0 = sb + OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  // rows landed / operand region free again / operand made, by chunk parity
  const uint32_t staged = bar(0), kq_free = bar(2), rdy_kq = bar(4);
  const uint32_t vstaged = bar(6), v_free = bar(7);
  const uint32_t rdy_s = bar(8), rdy_v = bar(9), rdy_p = bar(10);
  const uint32_t done_qk = bar(11), done_o = bar(12), done_kv = bar(13);
  const uint32_t acc_free = bar(14), drain = bar(15), vecs = bar(16);  // 16..19
  volatile uint32_t *slot = reinterpret_cast<volatile uint32_t *>(gb + OFF_BAR + 160);
  volatile int *fail = reinterpret_cast<volatile int *>(gb + OFF_BAR + 164);
  auto vec = [&](int it) { return reinterpret_cast<float *>(gb + OFF_VEC + (it & 3) * 2048); };
  auto rowexp = [&](int it) { return reinterpret_cast<int *>(gb + OFF_EXP + (it & 1) * 512); };
  auto lanef = [&](int it) { return reinterpret_cast<float *>(gb + OFF_LANE + (it & 3) * 1024); };

  // first token of a chunk whose v is not finite, by half and column
  auto badtok = [&](int it) {
    return reinterpret_cast<unsigned char *>(gb + OFF_BAD + (it & 3) * 256);
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, half = (warp >> 2) & 1;
  const int myrow = 32 * quad + lane;          // TMEM lane

  if (warp == kIssuer) tmem_alloc(sb + OFF_BAR + 160, 512);
  if (tid == 0) {
    const int count[20] = {1, 1, 1, 1, kGroup, kGroup, 1, 8, kGroup, kGroup,
                           kGroup, 1, 1, 1, kGroup, 1, 1, 1, 1, 1};
    for (int i = 0; i < 20; ++i) mbar_init(bar(i), count[i]);
    *fail = 0;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);

  if (warp < 8) {
    // ============================================ group A: state, V operands
    float s[kC];  // state rows dk = 64 half .. + 63 of column dv = myrow
    float *ps = reinterpret_cast<float *>(gb + OFF_PS);
    float2 *pv = reinterpret_cast<float2 *>(gb + OFF_PV);
    // the state operand of chunk `it`
    auto state_operand = [&](int it) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < kC; ++j) m = amax(m, s[j]);
      ps[128 * half + myrow] = m;
      bar_pair(quad);
      const int e = scale_exp(amax(m, ps[128 * (half ^ 1) + myrow]));
      const float f = pow2(e);
#pragma unroll
      for (int c0 = 0; c0 < kC; c0 += 16)
        put16<kLo>(tl + T_SOP, tl + T_SOP + 64, 64 * half + c0, s + c0, f);
      if (half == 0) lanef(it)[myrow] = pow2(-e);
      tmem_wait_st();
      signal_ready(rdy_s);
    };
    auto store_state = [&](float *dst) {
#pragma unroll
      for (int j = 0; j < kC; ++j) dst[(size_t)(kC * half + j) * kD + myrow] = s[j];
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
    for (Walk<kLocal> w(P); w.ok;) {
      const int it = w.it;
      if (w.first) {
        const size_t at = ((size_t)w.head * P.nseg + w.seg) * kD * kD;
        const float *src = P.nseg > 1 ? P.ws_state + at : P.S + at;
#pragma unroll
        for (int j = 0; j < kC; ++j)
          s[j] = kLocal ? 0.f : src[(size_t)(kC * half + j) * kD + myrow];
        if (!kLocal) state_operand(it);
      }
      // ---- V^T and (V f)^T operands, lane dv, K = t = 32 half .. + 31
      wait_bar(vstaged, it & 1, fail);
      wait_bar(vecs + 8 * (it & 3), (it >> 2) & 1, fail);
      const float *vc = vec(it);
      const int nv = w.valid() - 32 * half;  // of this thread's 32 tokens
      auto vload = [&](int j) -> float {
        const int t = 32 * half + j;
        if (kBf16) {
          const uint32_t h = *reinterpret_cast<const unsigned short *>(
              gb + OFF_V + t * 256 + 2 * myrow);
          return __uint_as_float(h << 16);
        }
        return *reinterpret_cast<const float *>(gb + OFF_V + t * 512 + 4 * myrow);
      };
      float ma = 0.f, mb = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float x = j < nv ? vload(j) : 0.f;
        ma = amax(ma, x);
        mb = amax(mb, x * vc[VF + 32 * half + j]);
      }
      // A value that is not finite must not reach the rows before it (its
      // weight there is 0, but 0 * inf is NaN): PV takes 0 for it, and the
      // output becomes NaN from its token on.
      int bad = kC;
      if (!kLocal && __float_as_int(ma) >= 0x7f800000) {
        ma = 0.f;
#pragma unroll 1
        for (int j = 31; j >= 0; --j) {
          const float x = j < nv ? vload(j) : 0.f;
          if (!isfinite(x))
            bad = 32 * half + j;
          else
            ma = amax(ma, x);
        }
      }
      if (!kLocal) badtok(it)[128 * half + myrow] = bad;
      pv[128 * half + myrow] = make_float2(ma, mb);
      bar_pair(quad);
      const float2 other = pv[128 * (half ^ 1) + myrow];
      const int ea = scale_exp(amax(ma, other.x)), eb = scale_exp(amax(mb, other.y));
      const float fa = pow2(ea), fb = pow2(eb);
      if (!kLocal) {
        // V's columns are free once the previous chunk's PV has read them
        if (it > 0) wait_bar(done_o, (it - 1) & 1, fail);
        fence_after_sync();
        if (half == 0) lanef(it)[128 + myrow] = pow2(-ea);
      }
#pragma unroll
      for (int c0 = 0; c0 < 32; c0 += 16) {
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = c0 + j < nv ? vload(c0 + j) : 0.f;
        const int t0 = 32 * half + c0;
        if (!kLocal) {
          float y[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = x[j];
          if (bad < kC)
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = isfinite(x[j]) ? x[j] : 0.f;
          put16<kLo>(tl + T_VOP, tl + T_VOP + 32, t0, y, fa);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= vc[VF + t0 + j];
        put16<true>(tl + T_WOP, tl + T_WOP + 32, t0, x, fb);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(v_free);
      tmem_wait_st();
      signal_ready(rdy_v);
      // ---- the state after the chunk
      const float gC = vc[VM], inv = pow2(-eb);
      wait_bar(done_kv, it & 1, fail);
      fence_after_sync();
#pragma unroll
      for (int c0 = 0; c0 < kC; c0 += 32) {
        uint32_t d[32];
        tmem_ld32_async(tl + T_D + 64 * half + c0, d);
        tmem_wait_ld(d);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          s[c0 + j] = fmaf(gC, s[c0 + j], __uint_as_float(d[j]) * inv);
      }
      if (w.last()) {
        const size_t hd = (size_t)w.head * kD * kD;
        if (kLocal)
          store_state(P.ws_state + ((size_t)w.head * P.nseg + w.seg) * kD * kD);
        else if (w.seg == P.nseg - 1)
          store_state(P.S + hd);
        if (kLocal) signal_ready(rdy_s);
      } else if (kLocal) {
        signal_ready(rdy_s);  // the KV columns are read
      } else {
        state_operand(it + 1);
      }
      w.next();
    }
  } else if (warp < 16) {
    // ======================================= group B: q, k rows, P, output
    const int bt = tid - kGroup;
    // [K; Q] operand of a chunk, in place: rows (bt >> 4) + 16 i, columns
    // 8 (bt & 15) .. + 7; rows 0-63 K, 64-127 Q
    auto convert = [&](const Walk<kLocal> &w) {
      const uint32_t reg = OFF_KQ + (w.it & 1) * kKQ;
      wait_bar(staged + 8 * (w.it & 1), (w.it >> 1) & 1, fail);
      constexpr int kRows = kLocal ? 4 : 8;
      const int swap = (bt >> 2) & 1, c0 = (bt & 15) * 8, nv = w.valid();
      float x[kRows][8];
      float sc[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = (bt >> 4) + 16 * i;
        if (kBf16) {
          const uint4 u = *reinterpret_cast<const uint4 *>(gb + reg + row * 256 + c0 * 2);
          const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[i][2 * j] = __uint_as_float(q[j] << 16);
            x[i][2 * j + 1] = __uint_as_float(q[j] & 0xffff0000u);
          }
        } else {
          const float *st = reinterpret_cast<const float *>(gb + reg) + row * 128 + c0;
          const float4 ya = *reinterpret_cast<const float4 *>(st + 4 * swap);
          const float4 yb = *reinterpret_cast<const float4 *>(st + 4 - 4 * swap);
          const float4 x0 = swap ? yb : ya, x1 = swap ? ya : yb;
          x[i][0] = x0.x; x[i][1] = x0.y; x[i][2] = x0.z; x[i][3] = x0.w;
          x[i][4] = x1.x; x[i][5] = x1.y; x[i][6] = x1.z; x[i][7] = x1.w;
        }
        if ((row & 63) >= nv)
#pragma unroll
          for (int j = 0; j < 8; ++j) x[i][j] = 0.f;
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = amax(m, x[i][j]);
#pragma unroll
        for (int d = 8; d; d >>= 1) m = amax(m, __shfl_xor_sync(0xffffffffu, m, d));
        const int e = scale_exp(m);
        sc[i] = pow2(e);
        if ((bt & 15) == 0) rowexp(w.it)[row] = e;
      }
      if (!kLocal && bt == 0)  // the o tile's last store has read it
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      bar_b();
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        put8<kLo>(gb, reg, 128, 128, (bt >> 4) + 16 * i, c0, x[i], sc[i]);
      signal_ready(rdy_kq + 8 * (w.it & 1));
    };
    Walk<kLocal> w(P);
    if (w.ok) convert(w);
    while (w.ok) {
      Walk<kLocal> nx = w;
      nx.next();
      if (kLocal) {
        if (nx.ok) convert(nx);
        w = nx;
        continue;
      }
      const int it = w.it;
      const float *vc = vec(it);
      // ---- P[t][s] = G e^{Gamma_t - Gamma_s}, s <= t (lanes 64-127: q rows)
      wait_bar(vecs + 8 * (it & 3), (it >> 2) & 1, fail);
      wait_bar(done_qk, it & 1, fail);
      fence_after_sync();
      if (quad >= 2) {
        const int t = myrow - kC, s0 = 32 * half;
        if (s0 <= 32 * (quad - 2)) {
          uint32_t r[32];
          tmem_ld32_async(tl + T_G + s0, r);
          tmem_wait_ld(r);
          const float at = vc[VA + t];
          float x[32];
          if (vc[VM + 1] != 0.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              x[j] = s0 + j <= t ? __uint_as_float(r[j]) * (at * vc[VB + s0 + j]) : 0.f;
          } else {
            const float gh = vc[VGH + t], gl = vc[VGL + t];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float d = (gh - vc[VGH + s0 + j]) + (gl - vc[VGL + s0 + j]);
              x[j] = s0 + j <= t
                         ? __uint_as_float(r[j]) * (at * vc[VB + s0 + j]) * exp2f(d)
                         : 0.f;
            }
          }
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 8)
            put8<kLo>(gb, OFF_P, kC, kC, t, s0 + c0, x + c0, 1.f);
        } else {
          const float z[8] = {};
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 8) put8<kLo>(gb, OFF_P, kC, kC, t, s0 + c0, z, 1.f);
        }
      }
      signal_ready(rdy_p);
      // ---- the next chunk's rows, under this one's products
      if (nx.ok) {
        convert(nx);
      } else {
        if (bt == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        bar_b();
      }
      // ---- o^T = cA QS + cB PV, lane dv, columns t = 32 half .. + 31
      wait_bar(done_o, it & 1, fail);
      fence_after_sync();
      {
        uint32_t qs[32], pvr[32];
        tmem_ld32_async(tl + T_QS + 32 * half, qs);
        tmem_ld32_async(tl + T_G + 32 * half, pvr);
        const float fs = lanef(it)[myrow], fv = lanef(it)[128 + myrow];
        tmem_wait_ld(qs);
        tmem_wait_ld(pvr);
        fence_before_sync();
        mbar_arrive(acc_free);
        unsigned char *ot = gb + OFF_O + 32 * half * kRow;
        const int bad = min((int)badtok(it)[myrow], (int)badtok(it)[128 + myrow]);
        const bool finite = bad >= kC;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int t = 32 * half + j;
          float y = fmaf(__uint_as_float(qs[j]) * fs, vc[VCA + t],
                         __uint_as_float(pvr[j]) * fv * vc[VCB + t]);
          if (!finite && t >= bad) y = __int_as_float(0x7fffffff);
          if (kBf16)
            *reinterpret_cast<__nv_bfloat16 *>(ot + j * 256 + 2 * myrow) = __float2bfloat16_rn(y);
          else
            *reinterpret_cast<float *>(ot + j * 512 + 4 * myrow) = y;
        }
      }
      fence_proxy_async();
      bar_b();
      const int nv = w.valid();
      if (nv == kC) {
        if (bt == 0) tma_store(&tm_o, w.vi, w.c * kC, w.b, sb + OFF_O);
      } else {  // a part of a chunk: only its rows
        constexpr int kVec = kRow / 16;
        for (int e = bt; e < nv * kVec; e += kGroup) {
          const int r = e / kVec, x = e % kVec;
          const size_t tok = (size_t)w.b * P.T + (size_t)w.c * kC + r;
          *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(P.o) +
                                     (tok * P.vh + w.vi) * kRow + x * 16) =
              *reinterpret_cast<const uint4 *>(gb + OFF_O + r * kRow + x * 16);
        }
      }
      w = nx;
    }
    if (!kLocal && bt == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (warp == kIssuer) {
    // =================================================== the issuing thread
    if (lane == 0) {
      for (Walk<kLocal> w(P); w.ok; w.next()) {
        const int it = w.it;
        const uint32_t kq = sb + OFF_KQ + (it & 1) * kKQ, ql = 32768u;
        wait_bar(rdy_kq + 8 * (it & 1), (it >> 1) & 1, fail);
        if (!kLocal) {
          if (it > 0) wait_bar(acc_free, (it - 1) & 1, fail);
          fence_after_sync();
          constexpr uint32_t id = idesc16(128, kC, 0);
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks) {
            const uint64_t h = kdesc(kq, 128, ks), l = kdesc(kq + ql, 128, ks);
            mma_bf16(tmem + T_G, h, h, id, ks > 0);
            if (kLo) {
              mma_bf16(tmem + T_G, h, l, id, 1u);
              mma_bf16(tmem + T_G, l, h, id, 1u);
            }
          }
          commit(done_qk);
          wait_bar(rdy_s, it & 1, fail);
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks) {
            // Q: rows 64-127 of the operand
            const uint64_t h = kdesc(kq + 8192u, 128, ks), l = kdesc(kq + ql + 8192u, 128, ks);
            const uint32_t a = tmem + T_SOP + 8u * ks;
            mma_bf16_ta(tmem + T_QS, a, h, id, ks > 0);
            if (kLo) {
              mma_bf16_ta(tmem + T_QS, a, l, id, 1u);
              mma_bf16_ta(tmem + T_QS, a + 64u, h, id, 1u);
            }
          }
        } else {
          // the KV columns are free once the state has taken the last product
          if (it > 0) wait_bar(rdy_s, (it - 1) & 1, fail);
        }
        wait_bar(rdy_v, it & 1, fail);
        fence_after_sync();
        {
          constexpr uint32_t id = idesc16(128, kD, 1);
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks) {
            const uint64_t h = mndesc(kq, 128, ks), l = mndesc(kq + ql, 128, ks);
            const uint32_t a = tmem + T_WOP + 8u * ks;
            mma_bf16_ta(tmem + T_D, a, h, id, ks > 0);
            mma_bf16_ta(tmem + T_D, a + 32u, h, id, 1u);
            if (kLo) mma_bf16_ta(tmem + T_D, a, l, id, 1u);
          }
        }
        commit(done_kv);
        commit(kq_free + 8 * (it & 1));
        if (!kLocal) {
          wait_bar(rdy_p, it & 1, fail);
          fence_after_sync();
          constexpr uint32_t id = idesc16(128, kC, 0);
          const uint32_t p = sb + OFF_P;
#pragma unroll
          for (int ks = 0; ks < kC / 16; ++ks) {
            const uint64_t h = kdesc(p, kC, ks), l = kdesc(p + 8192u, kC, ks);
            const uint32_t a = tmem + T_VOP + 8u * ks;
            mma_bf16_ta(tmem + T_G, a, h, id, ks > 0);
            if (kLo) {
              mma_bf16_ta(tmem + T_G, a, l, id, 1u);
              mma_bf16_ta(tmem + T_G, a + 32u, h, id, 1u);
            }
          }
          commit(done_o);
        }
      }
      commit(drain);  // arrives once every product issued above is done
    }
    __syncwarp();
  } else if (warp == kLoader) {
    // ===================================================== the copying warp
    if (lane == 0) {
      int it = 0;
      for (Walk<kLocal> w(P); w.ok; w.next()) {
        it = w.it;
        const uint32_t reg = sb + OFF_KQ + (it & 1) * kKQ, st = staged + 8 * (it & 1);
        if (it >= 2) wait_bar(kq_free + 8 * (it & 1), ((it - 2) >> 1) & 1, fail);
        mbar_expect(st, (kLocal ? 1u : 2u) * kC * kRow);
        tma_load(reg, &tm_k, w.vi / P.rep, w.c * kC, w.b, st);
        if (!kLocal) tma_load(reg + kC * kRow, &tm_q, w.vi / P.rep, w.c * kC, w.b, st);
        if (it >= 1) wait_bar(v_free, (it - 1) & 1, fail);
        mbar_expect(vstaged, kC * kRow);
        tma_load(sb + OFF_V, &tm_v, w.vi, w.c * kC, w.b, vstaged);
        ++it;
      }
      // nothing may still be copying into shared memory when the CTA ends
      // (the last chunk of either parity, and the last V rows)
      for (int j = it - 2; j < it; ++j)
        if (j >= 0) mbar_wait(staged + 8 * (j & 1), (j >> 1) & 1, kWaitLimit);
      if (it > 0) mbar_wait(vstaged, (it - 1) & 1, kWaitLimit);
    }
    __syncwarp();
  } else if (warp == kGates) {
    // ====================================================== decay vectors
    // Lane l has tokens l and l + 32.  exp2 of a double difference: its float
    // part, times 1 + ln 2 of the rest.
    auto ex2 = [](double x) {
      const float h = (float)x;
      const float l = (float)(x - (double)h);
      const float e = exp2f(h);
      return fmaf(e, l * 0.69314718f, e);
    };
    double total = 0.0;
    for (Walk<kLocal> w(P); w.ok; w.next()) {
      const int it = w.it, nv = w.valid();
      if (w.first) total = 0.0;
      const size_t base = P.g_head ? (size_t)w.vi
                                   : ((size_t)w.b * P.T + (size_t)w.c * kC) * P.vh + w.vi;
      const size_t step = P.g_head ? 0 : (size_t)P.vh;
      float ga = lane < nv ? __ldg(P.g + base + lane * step) : 0.f;
      float gc = lane + 32 < nv ? __ldg(P.g + base + (lane + 32) * step) : 0.f;
      // -inf as a decay that no float survives; NaN stays
      if (ga < -1e4f) ga = -1e4f;
      if (gc < -1e4f) gc = -1e4f;
      double da = (double)ga * 1.4426950408889634, dc = (double)gc * 1.4426950408889634;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double ya = __shfl_up_sync(0xffffffffu, da, off);
        const double yc = __shfl_up_sync(0xffffffffu, dc, off);
        if (lane >= off) {
          da += ya;
          dc += yc;
        }
      }
      dc += __shfl_sync(0xffffffffu, da, 31);
      const double end = __shfl_sync(0xffffffffu, dc, 31);
      total += end;
      float *vc = vec(it);
      const float wa = ex2(end - da), wc = ex2(end - dc);
      if (kLocal) {
        wait_bar(rdy_kq + 8 * (it & 1), (it >> 1) & 1, fail);
        const int *ex = rowexp(it);
        vc[VF + lane] = wa * pow2(-ex[lane]);
        vc[VF + lane + 32] = wc * pow2(-ex[lane + 32]);
        if (lane == 0) vc[VM] = ex2(end);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(vecs + 8 * (it & 3));
          if (w.last()) P.ws_decay[(size_t)w.head * P.nseg + w.seg] = total;
        }
        continue;
      }
      // growth: the largest Gamma_t - Gamma_s, s <= t (0 for decays)
      const float fa = (float)da, fc = (float)dc;
      float na = fa, nc = fc;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const float ya = __shfl_up_sync(0xffffffffu, na, off);
        const float yc = __shfl_up_sync(0xffffffffu, nc, off);
        if (lane >= off) {
          na = fminf(na, ya);
          nc = fminf(nc, yc);
        }
      }
      nc = fminf(nc, __shfl_sync(0xffffffffu, na, 31));
      float grow = fmaxf(fa - na, fc - nc), top = fmaxf(fa, fc), low = fminf(fa, fc);
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        grow = fmaxf(grow, __shfl_xor_sync(0xffffffffu, grow, off));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
      }
      const int ew = 22 + (int)ceilf(fminf(grow, 80.f));
      // one factor per row and column while their product cannot leave the
      // normal floats; otherwise an exponential per element
      const bool fac = top - low <= 115.f;
      const double mid = 0.5 * ((double)top + (double)low);
      const float ra = fac ? ex2(da - mid) : 1.f, rc = fac ? ex2(dc - mid) : 1.f;
      const float ca = fac ? ex2(mid - da) : 1.f, cc = fac ? ex2(mid - dc) : 1.f;
      const float Ga = ex2(da), Gc = ex2(dc);
      wait_bar(rdy_kq + 8 * (it & 1), (it >> 1) & 1, fail);
      const int *ex = rowexp(it);
      const int ka = ex[lane], kc = ex[lane + 32], qa = ex[64 + lane], qc = ex[96 + lane];
      int pa = ka, pc = kc;  // the smallest exponent (largest k row) up to t
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int ya = __shfl_up_sync(0xffffffffu, pa, off);
        const int yc = __shfl_up_sync(0xffffffffu, pc, off);
        if (lane >= off) {
          pa = min(pa, ya);
          pc = min(pc, yc);
        }
      }
      pc = min(pc, __shfl_sync(0xffffffffu, pa, 31));
      // where the two factors split: the smallest exponent of a finite row
      int ref = min(ka > -114 ? ka : 126, kc > -114 ? kc : 126);
#pragma unroll
      for (int off = 16; off; off >>= 1) ref = min(ref, __shfl_xor_sync(0xffffffffu, ref, off));
      // (exactly; 0 below the normal floats)
      auto p2 = [](int e) { return e < -126 ? 0.f : pow2(min(e, 127)); };
      vc[VA + lane] = ra * p2(pa - ref - ew);
      vc[VA + lane + 32] = rc * p2(pc - ref - ew);
      vc[VB + lane] = ca * p2(ref - ka);
      vc[VB + lane + 32] = cc * p2(ref - kc);
      vc[VF + lane] = wa * p2(-ka);
      vc[VF + lane + 32] = wc * p2(-kc);
      vc[VCA + lane] = P.scale * Ga * p2(-qa);
      vc[VCA + lane + 32] = P.scale * Gc * p2(-qc);
      vc[VCB + lane] = P.scale * p2(ew - qa - pa);
      vc[VCB + lane + 32] = P.scale * p2(ew - qc - pc);
      vc[VGH + lane] = fa;
      vc[VGH + lane + 32] = fc;
      vc[VGL + lane] = (float)(da - (double)fa);
      vc[VGL + lane + 32] = (float)(dc - (double)fc);
      if (lane == 0) {
        vc[VM] = ex2(end);
        vc[VM + 1] = fac ? 1.f : 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(vecs + 8 * (it & 3));
    }
    if (kLocal) {  // segments without a chunk: no decay
      Walk<kLocal> w(P);
      for (int u = blockIdx.x; u < P.units; u += gridDim.x) {
        w.u = u;
        w.decode();
        if (w.c >= w.c_hi && lane == 0) P.ws_decay[(size_t)w.head * P.nseg + w.seg] = 0.0;
      }
    }
  }

  if (warp == kIssuer) {
    if (lane == 0) mbar_wait(drain, 0, kWaitLimit);
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
  if (*fail) {
    // a wait ran out: everything this CTA was to write becomes NaN, so the
    // failure shows in the results as well as in the counter
    if (tid == 0) atomicAdd(&g_linattn_timeouts, 1u);
    const float nan = __int_as_float(0x7fffffff);
    Walk<kLocal> w(P);
    for (int u = blockIdx.x; u < P.units; u += gridDim.x) {
      w.u = u;
      w.decode();
      const size_t at = ((size_t)w.head * P.nseg + w.seg) * kD * kD;
      float *dst = kLocal ? P.ws_state + at : P.S + (size_t)w.head * kD * kD;
      for (int e = tid; e < kD * kD; e += kThreads) dst[e] = nan;
      const int t_end = kLocal ? 0 : min(w.n, w.c_hi * kC);
      for (int t = w.c * kC; t < t_end; ++t) {
        const size_t row = (((size_t)w.b * P.T + t) * P.vh + w.vi) * kRow;
        if (tid < (int)kRow / 4)
          *reinterpret_cast<uint32_t *>(static_cast<unsigned char *>(P.o) + row + 4 * tid) =
              0x7fffffffu;
      }
    }
  }
}

// Start states of the segments from their own sums: for each head, in order,
// slot i takes the state before segment i and the state moves on by the
// segment's decay and sum.  One thread per four state elements.
__global__ void __launch_bounds__(256)
    linattn_chain_kernel(const float *__restrict__ S, float *__restrict__ ws,
                         const double *__restrict__ decay, int nseg) {
  const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t head = e / (kD * kD / 4), x = e % (kD * kD / 4);
  float4 s = reinterpret_cast<const float4 *>(S)[e];
  float4 *w = reinterpret_cast<float4 *>(ws) + head * nseg * (kD * kD / 4) + x;
  for (int i = 0; i < nseg; ++i, w += kD * kD / 4) {
    if (i == nseg - 1) {
      *w = s;
      break;
    }
    const float4 d = *w;
    const double l = decay[head * nseg + i];
    const float h = (float)l, a0 = exp2f(h), a = fmaf(a0, (float)(l - (double)h) * 0.69314718f, a0);
    *w = s;
    s.x = fmaf(a, s.x, d.x);
    s.y = fmaf(a, s.y, d.y);
    s.z = fmaf(a, s.z, d.z);
    s.w = fmaf(a, s.w, d.w);
  }
}

// Segments per sequence.  One segment costs its chunks on the critical CTA;
// more segments run the KV pass too (about 0.6 of the main pass per chunk)
// and read and write a start state each (about 2 chunks).  The cheapest
// count by that model.
int plan(int B, int vh, int T) {
  const long long heads = (long long)B * vh;
  const int n = (T + kC - 1) / kC;
  int best = 1;
  double cost = 1e300;
  for (int s = 1; s <= 64 && s <= n; ++s) {
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

PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// [B][T][heads][128] rows as a 4-d tensor {128, heads, T, B}; a box is 64
// token rows of one head.  Rows past T read as zeros and are not written.
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

template <bool kBf16, bool kLocal>
cudaError_t launch(const CUtensorMap *m, const Args &a, cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(linattn_chunk_kernel<kBf16, kLocal>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  linattn_chunk_kernel<kBf16, kLocal>
      <<<(unsigned)min(a.units, kSms), kThreads, kSmemAlloc, stream>>>(m[0], m[1], m[2], m[3], a);
  return cudaGetLastError();
}

}  // namespace

size_t linattn_prefill_workspace_bytes(int B, int vh, int T, bool) {
  const size_t heads = (size_t)B * vh;
  const size_t nseg = (size_t)plan(B, vh, T);
  const size_t bytes = heads * nseg * (kD * kD * sizeof(float) + sizeof(double));
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
  a.nchunks = (L.M + kC - 1) / kC;
  CUtensorMap m[4];
  cudaError_t e;
  if ((e = rows_map(&m[0], L.q, bf16, L.kh, L.M, L.B)) != cudaSuccess) return e;
  if ((e = rows_map(&m[1], L.k, bf16, L.kh, L.M, L.B)) != cudaSuccess) return e;
  if ((e = rows_map(&m[2], L.v, bf16, L.vh, L.M, L.B)) != cudaSuccess) return e;
  if ((e = rows_map(&m[3], L.o, bf16, L.vh, L.M, L.B)) != cudaSuccess) return e;
  if (nseg > 1) {
    a.units = (int)(heads * (nseg - 1));
    e = bf16 ? launch<true, true>(m, a, stream) : launch<false, true>(m, a, stream);
    if (e != cudaSuccess) return e;
    linattn_chain_kernel<<<(unsigned)(heads * (kD * kD / 4 / 256)), 256, 0, stream>>>(
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
