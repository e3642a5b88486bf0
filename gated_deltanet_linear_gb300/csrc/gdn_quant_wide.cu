// Projections with 4-bit weights for many rows of x (gdn_quant.cu has the form
// for few): y^T = W x^T on tcgen05 tensor cores.
//
// A CTA takes 128 weight rows (the M of the product, one TMEM lane each), 32 or
// 64 rows of x (N) and, in a cluster, a slice of K, in stages of 128 elements:
//   all 16 warps   codes -> bf16 (exact), x -> bf16 (bf16 x as it is; fp32 x as
//                  the sum of three bf16 numbers, 24 bits, nothing to scale),
//                  into 128-byte-swizzled operand tiles in shared memory
//   one thread     the products of the stage, one accumulator for each group of
//                  the stage (W x1, then x2 and x3 onto it)
//   all 16 warps   two stages later: accumulator times the group's scale, added
//                  to fp32 sums in registers (lane = weight row)
// The products of a stage run under the conversion of the next one.  The
// elements of 8 codes are used in the order in which they unpack (0, 4, 1, 5,
// ...), on both sides.  The sums of a cluster's slices meet in the shared
// memory of the CTA that writes the rows of y, added in slice order: the same
// bits on every call.
//
// Bound by the latency of a stage (sums, conversion, loads, one barrier: 1700
// cycles, in which the smem traffic takes 800 and the issue slots 1100), then
// by start and exchange (6000 cycles a call).  64 rows of 5120 x 6144: bf16
// 19.3 us, fp32 35 us; mma.sync with 16 rows of x at a time took 54 us.

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <array>
#include <map>
#include <mutex>
#include <type_traits>

#include "gdn_internal.cuh"
#include "gdn_tc.cuh"

namespace cg = cooperative_groups;

namespace gdn {

__device__ unsigned int g_quant_timeouts = 0;

namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr int kRowsW = 128;   // weight rows of a CTA
constexpr int kStage = 128;   // k elements of a stage
constexpr uint32_t kWaitLimit = 1u << 24;
constexpr int kATile = kRowsW * kStage * 2;
constexpr int kScales = 4 * 4 * kRowsW * 4;  // of four stages, up to 4 groups each

template <bool kBf16, int kNC>
__host__ __device__ constexpr int b_tile() {  // all parts of x
  return (kBf16 ? 1 : 3) * kNC * kStage * 2;
}
template <bool kBf16, int kNC>
__host__ __device__ constexpr int smem_bytes() {
  // two stages, the sums received from the cluster (up to 8 slices of at most
  // ceil(kNC / c) rows of y), the scales of four stages, barriers, room to align
  return 2 * (kATile + b_tile<kBf16, kNC>()) + (kNC + 8) * kRowsW * 4 + kScales + 64 + 1024;
}

struct WideArgs {
  const void *x;
  const uint8_t *qw;
  const __half *sc;
  void *y;
  int rows, N, K, csize, stages;  // stages: of the whole of K
};

__device__ __forceinline__ void codes(uint32_t u, uint32_t (&r)[4]) {
  const __nv_bfloat162 m = __floats2bfloat162_rn(-136.f, -136.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the code with bit 3 flipped is c + 8, in the mantissa of 128: 136 + c
    const uint32_t v = ((u >> (4 * i)) & 0x000f000fu) ^ 0x43084308u;
    const __nv_bfloat162 d = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&v), m);
    r[i] = *reinterpret_cast<const uint32_t *>(&d);
  }
}

template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[kN]) {
  if constexpr (kN == 16) {
    tmem_ld16(taddr, r);
  } else {
    uint32_t u[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(u[i]);
  }
}

template <bool kBf16, int kNC, int kGroup>
__global__ void __launch_bounds__(kThreads, 1) quant_wide_kernel(const WideArgs P) {
  using T = typename std::conditional<kBf16, __nv_bfloat16, float>::type;
  constexpr int kGroups = kStage / kGroup;        // of a stage
  constexpr int kTerms = kBf16 ? 1 : 3;
  constexpr int kCols = kNC / 4;                  // rows of y of a warp
  constexpr int kParts = kNC * (kStage / 8) / kThreads;  // 8-element parts of x a thread
  constexpr int kBTile = kNC * kStage * 2;
  constexpr uint32_t kTmem = 2 * kGroups * kNC;   // columns: 64 .. 512
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  unsigned char *gb = smem_raw + (sb - raw);
  constexpr uint32_t kStageBytes = kATile + kTerms * kBTile;
  float *recv = reinterpret_cast<float *>(gb + 2 * kStageBytes);  // [slice][row of y][weight row]
  // scales [stage & 3][group][weight row]
  float *scl = recv + (kNC + 8) * kRowsW;
  const uint32_t bar = sb + 2 * kStageBytes + (kNC + 8) * kRowsW * 4 + kScales;  // 2 mbarriers
  volatile uint32_t *slot = reinterpret_cast<volatile uint32_t *>(gb + (bar - sb) + 16);

  const cg::cluster_group cl = cg::this_cluster();
  const int csize = P.csize, crank = csize > 1 ? (int)cl.block_rank() : 0;
  const int n0 = (int)((unsigned)blockIdx.x / (unsigned)csize) * kRowsW;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, part = warp >> 2;

  if (warp == 0) tmem_alloc(bar + 16, kTmem);
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
  }
  // behind the kernel before it: nothing is read or written before it has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  fence_before_sync();
  if (csize > 1)
    cl.sync();  // every CTA's shared memory is there
  else
    __syncthreads();
  fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);

  const int s_lo = (int)((long long)P.stages * crank / csize);
  const int ns = (int)((long long)P.stages * (crank + 1) / csize) - s_lo;
  const int groups = P.K / kGroup;
  const size_t wrow = (size_t)P.K / 2;
  // this thread's piece of a stage: 32 codes of weight row tid >> 2 and, of that
  // row, the scale of group `piece` (rows behind the last one: the last one's).
  // The scales go through shared memory to the threads that keep a row's sums:
  // a load of 32 rows' scales by each of them took as long as the conversion
  // (32 lines a request).
  const int arow = tid >> 2, piece = tid & 3;
  const uint8_t *wp = P.qw + (size_t)min(n0 + arow, P.N - 1) * wrow + 16 * piece;
  const __half *sp = P.sc + (size_t)min(n0 + arow, P.N - 1) * groups;

  bool failed = false;
  uint32_t done = 0;  // stages issued so far, over all passes
  for (int r0 = 0; r0 < P.rows; r0 += kNC) {
    const int nr = min(kNC, P.rows - r0);
    float acc[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
    // Two stages of this slice in registers, ahead of use.
    uint4 w[2];
    float xv[2][kParts][8];
    __half sn[2];
    const T *xp[kParts];  // this thread's parts of x, nullptr behind the last row
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const int e = tid + i * kThreads, r = e >> 4;
      xp[i] = r < nr ? static_cast<const T *>(P.x) + (size_t)(r0 + r) * P.K + 8 * (e & 15)
                     : nullptr;
    }
    auto fetch = [&](int u, int s) {
      const int k0 = (s_lo + s) * kStage;
      // (a group behind the last one has zeros of x against any scale)
      if (piece < kGroups) sn[u] = __ldg(sp + min((s_lo + s) * kGroups + piece, groups - 1));
      w[u] = make_uint4(0, 0, 0, 0);
      if (k0 + 32 * piece < P.K) w[u] = __ldg(reinterpret_cast<const uint4 *>(wp + k0 / 2));
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const bool on = xp[i] != nullptr && k0 + 8 * (tid & 15) < P.K;
        const T *p = xp[i] + k0;
        const uint4 z = make_uint4(0, 0, 0, 0);
        const uint4 a = on ? __ldg(reinterpret_cast<const uint4 *>(p)) : z;
        const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[u][i][j] = __uint_as_float(q[j]);  // bf16: two to a word
        if constexpr (!kBf16) {
          const uint4 b = on ? __ldg(reinterpret_cast<const uint4 *>(p) + 1) : z;
          const uint32_t v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) xv[u][i][4 + j] = __uint_as_float(v[j]);
        }
      }
    };
    // Stage counts run on over the passes (barriers and buffers go by them); a
    // pass starts with both buffers free.
    const uint32_t base = done;
    if (ns > 0) fetch(0, 0);
    if (ns > 1) fetch(1, 1);
    for (int s0 = 0; s0 < ns + 2; s0 += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int s = s0 + u;
        if (s >= 2 && s < ns + 2) {
          // stage s - 2: its buffers are free, its accumulators full
          const uint32_t before = base + (uint32_t)(s - 2);  // index over all passes
          failed |= !mbar_wait(bar + 8 * (before & 1), (before >> 1) & 1u, kWaitLimit);
          fence_after_sync();
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            float d[kCols];
            tmem_ld<kCols>(tmem + ((uint32_t)(32 * quad) << 16) +
                               (uint32_t)(((before & 1) * kGroups + g) * kNC + part * kCols),
                           d);
            const float f = scl[((before & 3) * 4 + g) * kRowsW + 32 * quad + lane];
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = fmaf(f, d[i], acc[i]);
          }
        }
        if (s >= ns) continue;
        const uint32_t at = base + (uint32_t)s;
        unsigned char *A = gb + (at & 1) * kStageBytes, *B = A + kATile;
        if (piece < kGroups) scl[((at & 3) * 4 + piece) * kRowsW + arow] = __half2float(sn[u]);
        {
          const uint32_t word[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // (two pieces of a row lie in tiles that share banks: other order)
            const bool odd = piece >> 1;
            uint32_t r[4];
            codes(odd ? word[i ^ 2] : word[i], r);
            *reinterpret_cast<uint4 *>(
                A + sw128_off(kRowsW, arow, 32 * piece + 8 * (odd ? i ^ 2 : i), 2)) =
                make_uint4(r[0], r[1], r[2], r[3]);
          }
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const int e = tid + i * kThreads;
          unsigned char *dst = B + sw128_off(kNC, e >> 4, 8 * (e & 15), 2);
          float(&x)[8] = xv[u][i];
          if constexpr (kBf16) {
            const uint32_t q[4] = {__float_as_uint(x[0]), __float_as_uint(x[1]),
                                   __float_as_uint(x[2]), __float_as_uint(x[3])};
            *reinterpret_cast<uint4 *>(dst) =
                make_uint4(__byte_perm(q[0], q[2], 0x5410), __byte_perm(q[0], q[2], 0x7632),
                           __byte_perm(q[1], q[3], 0x5410), __byte_perm(q[1], q[3], 0x7632));
          } else {
#pragma unroll
            for (int term = 0; term < 3; ++term, dst += kBTile) {
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                // (cut off, so no finite element becomes infinite; the third
                // part is exact: 3 x 8 bits)
                const uint32_t p = __float_as_uint(x[j]), q = __float_as_uint(x[j + 4]);
                o[j] = __byte_perm(p, q, 0x7632);
                x[j] -= __uint_as_float(p & 0xffff0000u);
                x[j + 4] -= __uint_as_float(q & 0xffff0000u);
              }
              *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        if (s + 2 < ns) fetch(u, s + 2);
        fence_proxy_async();
        fence_before_sync();
        __syncthreads();
        if (warp == 0) {
          fence_after_sync();
          const uint32_t one = elect();
          const uint32_t a = sb + (at & 1) * kStageBytes, b = a + kATile;
          constexpr uint32_t id = idesc(kFmtBF16, kRowsW, kNC);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const uint32_t d = tmem + (uint32_t)(((at & 1) * kGroups + g) * kNC);
#pragma unroll
            for (int term = 0; term < kTerms; ++term)
#pragma unroll
              for (int k = 0; k < kGroup / 16; ++k) {
                const int ks = g * (kGroup / 16) + k;
                mma_ss(one, d, desc_kstep(a, kRowsW, ks), desc_kstep(b + term * kBTile, kNC, ks),
                       id, term > 0 || k > 0);
              }
          }
          commit_one(one, bar + 8 * (at & 1));
        }
      }
    }
    done = base + (uint32_t)ns;

    if (failed) {
      // a wait ran out: the results become NaN
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = __int_as_float(0x7fffffff);
    }
    const int n = n0 + 32 * quad + lane;
    auto put = [&](int col, float v) {
      if (n >= P.N || col >= nr) return;
      const size_t out = (size_t)(r0 + col) * P.N + n;
      if (kBf16)
        static_cast<__nv_bfloat16 *>(P.y)[out] = __float2bfloat16_rn(v);
      else
        static_cast<float *>(P.y)[out] = v;
    };
    if (csize == 1) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) put(part * kCols + i, acc[i]);
    } else {
      // rank c adds up rows c * per .. of y
      const int per = (kNC + csize - 1) / csize;
      int to = (unsigned)(part * kCols) / (unsigned)per, c = part * kCols - to * per;
      const int at = crank * per * kRowsW + 32 * quad + lane;
      float *dst = cl.map_shared_rank(recv, to) + at;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        dst[c * kRowsW] = acc[i];
        if (++c == per && i + 1 < kCols) {
          c = 0;
          dst = cl.map_shared_rank(recv, ++to) + at;
        }
      }
      cl.sync();
      // (4 columns a time, one by a group of four warps; 32 rows a warp)
      const float *src = recv + 32 * quad + lane;
#pragma unroll 2
      for (int c = part; c < per; c += 4) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < csize) v[q] = src[(q * per + c) * kRowsW];
        float sum = v[0];
#pragma unroll
        for (int q = 1; q < 8; ++q)
          if (q < csize) sum += v[q];
        if (crank * per + c < kNC) put(crank * per + c, sum);
      }
      if (r0 + kNC < P.rows) cl.sync();  // read before the next pass writes
    }
  }
  if (failed) atomicAdd(&g_quant_timeouts, 1u);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, kTmem);
}

// Clusters of 1 .. 8 CTAs of this size that the current device runs at once
// (asked once per device).
cudaError_t cluster_counts(std::array<int, 8> &most) {
  static std::mutex lock;
  static std::map<int, std::array<int, 8>> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> hold(lock);
  auto it = known.find(dev);
  if (it == known.end()) {
    const auto kernel = quant_wide_kernel<false, 64, 128>;
    const int bytes = smem_bytes<false, 64>();
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    std::array<int, 8> n;
    for (int c = 1; c <= 8; ++c) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(c);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = bytes;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = c;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n[c - 1], kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (n[c - 1] < 1) n[c - 1] = 1;
    }
    it = known.emplace(dev, n).first;
  }
  most = it->second;
  return cudaSuccess;
}

template <bool kBf16, int kNC, int kGroup>
cudaError_t launch(const WideArgs &a, int tiles, cudaStream_t stream) {
  const auto kernel = quant_wide_kernel<kBf16, kNC, kGroup>;
  constexpr int bytes = smem_bytes<kBf16, kNC>();
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * a.csize));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.csize;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.csize > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool kBf16, int kNC>
cudaError_t by_group(int group, const WideArgs &a, int tiles, cudaStream_t stream) {
  return group == 128  ? launch<kBf16, kNC, 128>(a, tiles, stream)
         : group == 64 ? launch<kBf16, kNC, 64>(a, tiles, stream)
                       : launch<kBf16, kNC, 32>(a, tiles, stream);
}

}  // namespace

cudaError_t launch_quant_linear_wide(const void *x, const unsigned char *qw, const void *scales,
                                     void *y, int rows, int N, int K, int group, bool bf16,
                                     cudaStream_t stream) {
  std::array<int, 8> most;
  const cudaError_t e = cluster_counts(most);
  if (e != cudaSuccess) return e;
  const int tiles = (N + kRowsW - 1) / kRowsW, stages = (K + kStage - 1) / kStage;
  // Slices of K: the waves of clusters times a CTA's stages, and about 6 stages
  // for a cluster's barriers and sums.
  int csize = 1;
  double best = 1e300;
  for (int c = 1; c <= 8 && c <= stages; ++c) {
    const int waves = (tiles + most[c - 1] - 1) / most[c - 1];
    const double cost = (double)waves * ((stages + c - 1) / c + 4 + (c > 1 ? 6 : 0));
    if (cost < best) {
      best = cost;
      csize = c;
    }
  }
  const WideArgs a{x, qw, static_cast<const __half *>(scales), y, rows, N, K, csize, stages};
  if (bf16)
    return rows <= 32 ? by_group<true, 32>(group, a, tiles, stream)
                      : by_group<true, 64>(group, a, tiles, stream);
  return rows <= 32 ? by_group<false, 32>(group, a, tiles, stream)
                    : by_group<false, 64>(group, a, tiles, stream);
}

cudaError_t quant_timeouts(unsigned int *count) {
  return cudaMemcpyFromSymbol(count, g_quant_timeouts, sizeof(unsigned int));
}

}  // namespace gdn
