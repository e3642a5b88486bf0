// Token-serial linear attention with a decay for each head, for sm_103a
// (decode, M-token verify).
//
// What it computes (per sequence b, value head vi, key head hh = vi / rep,
// token m):
//     S = exp(g) S + k v^T;   o = scale S^T q.
// The delta rule of gdn_decode.cu without its correction: nothing of the
// state has to be reduced before it is updated, so a token is one pass of
// multiply-adds over registers and the only reduction is o's.
//
// Work split.  A CTA of 4 warps takes a 32-column group of a head (16 KB of
// the 64 KB state), so that one sequence of 48 heads still gives every SM
// work.  Warp w has key rows 32w .. 32w+31; lane = 8 rg + cl has rows
// 32w + 8 rg .. + 7 and columns 4 cl .. 4 cl + 3 of the group: one warp
// request covers four whole 128-byte row segments, and a lane's q and k are
// 8 consecutive elements.  The 8 x 4 block stays in registers for all M
// tokens: the state is read once and written once per launch.  A lane keeps
// one of its 4 sums of o in the reduction over the row groups (3 shuffles
// instead of 8); the warps' sums meet in shared memory, one barrier for every
// 8 tokens.
//
// Arithmetic in packed pairs (rows 2 i and 2 i + 1 of a column): half the
// instructions of the 32 elements of a lane, k and q as they lie in shared
// memory.  (8 tokens x 64 x 48 heads 111 -> 95 us; 64 registers at 8 CTAs an SM,
// 80 at 6 took 109.)
//
// Determinism.  Every product and sum is an explicit round-to-nearest
// operation in a fixed tree (a lane's even rows and odd rows in order, the row groups
// (0 + 1) + (2 + 3), the warps (0 + 2) + (1 + 3)), so M tokens in one launch
// give the bits of M launches.
//
// Bound by HBM: 128 KB of state per head against three FP32 lane operations
// per state element and token.  64 sequences x 48 heads: one token 58.4 us bf16
// (405 MB, 103 % of the copy rate with what stays in L2; DRAM moves 6.0 TB/s, 90 %),
// 4 tokens 69 us bf16, 77 fp32, 8 tokens 89 and 94 us, where a CTA's
// phases (state in, 8 tokens of dependent sums, state out) overlap less.

#include <cuda_bf16.h>

#include "gdn_internal.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBlk = 8;  // tokens between barriers

__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}

__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
  const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
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
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t *>(&a);
  u.y = *reinterpret_cast<const uint32_t *>(&b);
  *reinterpret_cast<uint2 *>(p) = u;
}

__device__ __forceinline__ float4 ld_state(const float *p) {
  float4 v;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void st_state(float *p, const float4 &v) {
  asm volatile("st.global.L1::no_allocate.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// Token inputs of a block of tokens in shared memory, as fp32 (several tokens:
// converted once for the CTA's four warps, and read again without the latency
// of a cache miss).
struct Staged {
  float k[kBlk][kDim], q[kBlk][kDim], v[kBlk][32], a[kBlk];
};

// kMulti: more than one token: token inputs are staged 8 at a time.  One token:
// each lane reads its own, beside the state's loads.
template <typename T, bool kMulti>
__global__ void __launch_bounds__(128, kMulti ? 8 : 5)
    linattn_steps_kernel(const LinattnArgs P) {
  __shared__ float part[2][kBlk][4][32];
  __shared__ __align__(16) Staged st[1];
  // behind the kernel before it: nothing is read or written before that
  // kernel has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.x >> 2, cg = blockIdx.x & 3;
  const int b = head / P.vh, vi = head % P.vh, hh = vi / P.rep;
  const int n = P.M;
  const int row = 32 * warp + 8 * (lane >> 3);
  const int cl = 4 * (lane & 7), col = 32 * cg + cl;
  const size_t blk = (size_t)row * kDim + col;  // of the state

  const size_t tok0 = (size_t)b * P.M;
  const T *qp = static_cast<const T *>(P.q) + (tok0 * P.kh + hh) * kDim;
  const T *kp = static_cast<const T *>(P.k) + (tok0 * P.kh + hh) * kDim;
  const T *vp = static_cast<const T *>(P.v) + (tok0 * P.vh + vi) * kDim + 32 * cg;
  T *op = static_cast<T *>(P.o) + (tok0 * P.vh + vi) * kDim + 32 * cg;
  const float *gp = P.g + (P.g_head ? (size_t)vi : tok0 * P.vh + vi);
  const size_t qk_step = (size_t)P.kh * kDim, v_step = (size_t)P.vh * kDim;
  const size_t g_step = P.g_head ? 0 : P.vh;

  F2 s[4][4];  // rows 2 i and 2 i + 1 of a column
  {
    const float *Sp = P.S_in + (size_t)head * kDim * kDim + blk;
    float4 r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = ld_state(Sp + i * kDim);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i][0] = pack(r[2 * i].x, r[2 * i + 1].x);
      s[i][1] = pack(r[2 * i].y, r[2 * i + 1].y);
      s[i][2] = pack(r[2 * i].z, r[2 * i + 1].z);
      s[i][3] = pack(r[2 * i].w, r[2 * i + 1].w);
    }
  }
  // One token: S = a S + k v^T, and this lane's share of S^T q into part[j].
  const bool up8 = lane & 8, up16 = lane & 16;
  // the column of the group whose sum this lane ends up with
  const int mine = cl + 2 * (up8 ? 1 : 0) + (up16 ? 1 : 0);
  auto token = [&](const F2 (&k)[4], const F2 (&q)[4], const float (&v)[4], float a,
                   float (&sums)[4][32]) {
    float acc[4];
    const F2 aa = pack(a, a);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const F2 vv = pack(v[c], v[c]);
      F2 t = 0ull;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i][c] = fma2(aa, s[i][c], mul2(k[i], vv));
        t = fma2(s[i][c], q[i], t);
      }
      const float2 u = unpack(t);
      acc[c] = __fadd_rn(u.x, u.y);
    }
    float k0 = up8 ? acc[2] : acc[0], k1 = up8 ? acc[3] : acc[1];
    k0 = __fadd_rn(k0, __shfl_xor_sync(kFull, up8 ? acc[0] : acc[2], 8));
    k1 = __fadd_rn(k1, __shfl_xor_sync(kFull, up8 ? acc[1] : acc[3], 8));
    sums[warp][mine] = __fadd_rn(up16 ? k1 : k0, __shfl_xor_sync(kFull, up16 ? k0 : k1, 16));
  };
  auto state_to = [&](float *p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack(s[i][0]), y = unpack(s[i][1]), z = unpack(s[i][2]),
                   w = unpack(s[i][3]);
      st_state(p + blk + 2 * i * kDim, make_float4(x.x, y.x, z.x, w.x));
      st_state(p + blk + (2 * i + 1) * kDim, make_float4(x.y, y.y, z.y, w.y));
    }
  };
  // The sums of nb tokens from m0 on, from the four warps' parts.
  auto output = [&](int m0, int nb, float (&p)[kBlk][4][32]) {
    if (tid < 8 * nb) {
      const int j = tid >> 3, c = 4 * (tid & 7);
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[e] = __fmul_rn(P.scale, __fadd_rn(__fadd_rn(p[j][0][c + e], p[j][2][c + e]),
                                            __fadd_rn(p[j][1][c + e], p[j][3][c + e])));
      store4(op + (m0 + j) * v_step + c, y);
    }
  };
  if (!kMulti) {
    float f[8], v[4];
    F2 k[4], q[4];
    load8(kp + row, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = pack(f[2 * i], f[2 * i + 1]);
    load8(qp + row, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pack(f[2 * i], f[2 * i + 1]);
    load4(vp + cl, v);
    token(k, q, v, expf(__ldg(gp)), part[0][0]);
    if (P.ckpt) state_to(P.ckpt + (size_t)head * kDim * kDim);
    __syncthreads();
    output(0, 1, part[0]);
  } else {
    int buf = 0;
    for (int m0 = 0; m0 < n; m0 += kBlk, buf ^= 1) {
      const int nb = min(kBlk, n - m0);
      // (the last block's inputs are read: every warp has passed the barrier
      // behind its tokens)
      for (int e = tid; e < nb * 36; e += 128) {  // 8 elements each: 16 k, 16 q, 4 v
        const int j = e / 36, x = e - 36 * j;
        float f[8];
        if (x < 16)
          load8(kp + (m0 + j) * qk_step + 8 * x, f);
        else if (x < 32)
          load8(qp + (m0 + j) * qk_step + 8 * (x - 16), f);
        else
          load8(vp + (m0 + j) * v_step + 8 * (x - 32), f);
        float *d = x < 16 ? &st->k[j][8 * x] : x < 32 ? &st->q[j][8 * (x - 16)]
                                                      : &st->v[j][8 * (x - 32)];
        *reinterpret_cast<float4 *>(d) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(d + 4) = make_float4(f[4], f[5], f[6], f[7]);
      }
      if (tid < nb) st->a[tid] = expf(__ldg(gp + (m0 + tid) * g_step));
      __syncthreads();
#pragma unroll 1  // (unrolled, it took 3 % longer)
      for (int j = 0; j < nb; ++j) {
        F2 k[4], q[4];
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&st->k[j][row + 2 * i]);
          const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(&st->q[j][row + 2 * i]);
          k[i] = x.x; k[i + 1] = x.y;
          q[i] = y.x; q[i + 1] = y.y;
        }
        const float4 z = *reinterpret_cast<const float4 *>(&st->v[j][cl]);
        v[0] = z.x; v[1] = z.y; v[2] = z.z; v[3] = z.w;
        token(k, q, v, st->a[j], part[buf][j]);
        if (P.ckpt)
          state_to(P.ckpt + (((size_t)(m0 + j) * P.B * P.vh) + head) * kDim * kDim);
      }
      __syncthreads();
      // (the other buffer is written next; this one again only after the
      // barriers of the next block, which follow these reads)
      output(m0, nb, part[buf]);
    }
  }
  state_to(P.S_out + (size_t)head * kDim * kDim);
}

}  // namespace

cudaError_t launch_linattn_steps(const LinattnArgs &P, bool bf16,
                                 cudaStream_t stream) {
  const size_t blocks = (size_t)P.B * P.vh * 4;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffull) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (P.M == 1)
    return bf16 ? cudaLaunchKernelEx(&cfg, linattn_steps_kernel<__nv_bfloat16, false>, P)
                : cudaLaunchKernelEx(&cfg, linattn_steps_kernel<float, false>, P);
  return bf16 ? cudaLaunchKernelEx(&cfg, linattn_steps_kernel<__nv_bfloat16, true>, P)
              : cudaLaunchKernelEx(&cfg, linattn_steps_kernel<float, true>, P);
}

}  // namespace gdn
