// Projections with 4-bit weights for many rows of x (gdn_quant.cu has the form
// for few): y^T = W x^T on tcgen05 tensor cores.
//
// A CTA takes 128 weight rows (the M of the product, one TMEM lane each), 32 or
// 64 rows of x (N) and, in a cluster, a slice of K, in stages of 128 elements:
//   copy engine    codes (64 bytes of each row), and bf16 rows of x straight into
//                  128-byte-swizzled operand tiles, four stages ahead
//   16 warps       codes -> bf16 (exact), 32 of a row a thread, into TMEM: the A
//                  operand (through shared memory, its writes and the products'
//                  reads of it were two thirds of the traffic there); fp32 x ->
//                  three bf16 parts (3 x 8 bits, nothing to scale) into operand
//                  tiles
//   one thread     the products of the stage, one accumulator for each group of
//                  the stage (W x3, then x2 and x1 onto it)
//   16 warps       two stages later: accumulator times the group's scale, added
//                  to fp32 sums in registers (lane = weight row)
// The products of a stage run under the conversion of the next one.  The sums of
// a cluster's slices meet in the shared memory of the CTA that writes the rows of
// y, added in slice order: the same bits on every call.
//
// Bound by the chain of a stage (sums 450 cycles, unpacking 700, with 12 of its 16
// operations for 8 codes on the half-rate integer pipe, one barrier; 1500 in
// all), then by start and exchange (6000 cycles a call).  64 rows of 5120 x 6144:
// bf16 18.9 us (A through shared memory 19.3), fp32 28.7 (35.4); mma.sync with 16
// rows of x at a time took 54 us.  More rows go through the weights again for every
// 64: 512 rows 138 us (fp32 219), 4096 rows 1090 (1740).

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <array>
#include <map>
#include <mutex>
#include <type_traits>

#include "gdn_internal.cuh"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"

namespace cg = cooperative_groups;

namespace gdn {

__device__ unsigned int g_quant_timeouts = 0;

namespace {

using namespace tc;

constexpr int kThreads = 512;
constexpr int kRowsW = 128;   // weight rows of a CTA
constexpr int kStage = 128;   // k elements of a stage
constexpr uint32_t kWaitLimit = 1u << 24;
constexpr int kCodes = kRowsW * kStage / 2;  // bytes of a stage's codes
constexpr int kRing = 4;      // stages on their way
constexpr int kScales = 4 * 4 * kRowsW * 4;  // of four stages, up to 4 groups each

// Rows of x in shared memory: bf16 in the ring, fp32 the parts of two stages.
template <bool kBf16, int kNC>
__host__ __device__ constexpr int x_bytes() {
  return (kBf16 ? kRing : 2 * 3) * kNC * kStage * 2;
}
template <bool kBf16, int kNC>
__host__ __device__ constexpr int smem_bytes() {
  // codes, x, the sums received from the cluster (up to 8 slices of at most
  // ceil(kNC / c) rows of y), scales, barriers, room to align; and so much that
  // an SM has one CTA: CTAs of two clusters (on two streams) that hold TMEM on
  // one SM and wait for it on another would wait for each other
  constexpr int used =
      kRing * kCodes + x_bytes<kBf16, kNC>() + (kNC + 8) * kRowsW * 4 + kScales + 64 + 1024;
  return used > 118 * 1024 ? used : 118 * 1024;
}

struct WideArgs {
  const void *x;
  const uint8_t *qw;
  const __half *sc;
  void *y;
  int rows, N, K, csize, stages;  // stages: of the whole of K
};

// The 8 codes of a word, as four registers of two bf16 each, in order.
__device__ __forceinline__ void codes(uint32_t u, uint32_t *r) {
  const __nv_bfloat162 m = __floats2bfloat162_rn(-136.f, -136.f);
  uint32_t p[4];  // elements (0, 4), (1, 5), (2, 6), (3, 7)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the code with bit 3 flipped is c + 8, in the mantissa of 128: 136 + c
    const uint32_t v = ((u >> (4 * i)) & 0x000f000fu) ^ 0x43084308u;
    const __nv_bfloat162 d = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&v), m);
    p[i] = *reinterpret_cast<const uint32_t *>(&d);
  }
  r[0] = __byte_perm(p[0], p[1], 0x5410);
  r[1] = __byte_perm(p[2], p[3], 0x5410);
  r[2] = __byte_perm(p[0], p[1], 0x7632);
  r[3] = __byte_perm(p[2], p[3], 0x7632);
}

__device__ __forceinline__ void copy2d(uint32_t smem, const CUtensorMap *map, int x, int y,
                                       uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}

// 8 or 16 TMEM columns of this thread's lane; tcgen05.wait::ld before use.
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&u)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t (&u)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]),
        "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(taddr));
}

template <bool kBf16, int kNC, int kGroup>
__global__ void __launch_bounds__(kThreads, 1)
    quant_wide_kernel(const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_x, const WideArgs P) {
  constexpr int kGroups = kStage / kGroup;        // of a stage
  constexpr int kTerms = kBf16 ? 1 : 3;
  constexpr int kCols = kNC / 4;                  // rows of y of a warp
  constexpr int kParts = kNC * (kStage / 8) / kThreads;  // 8-element parts of x a thread
  constexpr int kBTile = kNC * kStage * 2;
  // TMEM columns: accumulators of two stages (of one, where two do not fit: a
  // stage's products are then waited for before the next one's), then the codes
  // of two
  constexpr int kLag = 2 * kGroups * kNC + 128 > 512 ? 1 : 2;
  constexpr uint32_t kAcc = kLag * kGroups * kNC, kTmem = kAcc + 128 > 256 ? 512 : 256;
  static_assert(kAcc + 128 <= 512, "TMEM");
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  unsigned char *gb = smem_raw + (sb - raw);
  constexpr uint32_t kX0 = kRing * kCodes, kEnd = kX0 + x_bytes<kBf16, kNC>();
  float *recv = reinterpret_cast<float *>(gb + kEnd);  // [slice][row of y][weight row]
  // scales [stage & 3][group][weight row]
  float *scl = recv + (kNC + 8) * kRowsW;
  // mbarriers: products done (by stage & 1), copies landed (by stage & 3)
  const uint32_t bar = sb + kEnd + (kNC + 8) * kRowsW * 4 + kScales, full = bar + 16;
  volatile uint32_t *slot = reinterpret_cast<volatile uint32_t *>(gb + (bar - sb) + 48);

  const cg::cluster_group cl = cg::this_cluster();
  const int csize = P.csize, crank = csize > 1 ? (int)cl.block_rank() : 0;
  const int n0 = (int)((unsigned)blockIdx.x / (unsigned)csize) * kRowsW;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, part = warp >> 2;

  if (warp == 0) tmem_alloc(bar + 48, kTmem);
  if (tid == 0) {
    for (int i = 0; i < 2 + kRing; ++i) mbar_init(bar + 8 * i, 1);
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
  // This thread's codes of a stage: 32 of the weight row of its TMEM lane (piece
  // `part`).  Scales are loaded by four threads to a row, coalesced, and go
  // through shared memory to the threads that keep the row's sums (rows behind
  // the last one: the last one's).
  const int row = 32 * quad + lane, srow = tid >> 2, piece = tid & 3;
  const __half *sp = P.sc + (size_t)min(n0 + srow, P.N - 1) * groups;
  const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
  const unsigned char *wp = gb + row * 64 + ((part ^ (row >> 1 & 3)) << 4);

  bool failed = false;
  uint32_t done = 0;  // stages issued so far, over all passes
  for (int r0 = 0; r0 < P.rows; r0 += kNC) {
    const int nr = min(kNC, P.rows - r0);
    float acc[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
    // Stage counts run on over the passes (barriers and buffers go by them); a
    // pass starts with all buffers free.
    const uint32_t base = done;
    // codes, and bf16 rows of x, of stage s
    auto copy = [&](int s) {
      const uint32_t t = base + (uint32_t)s, m = full + 8 * (t & 3);
      const int k0 = (s_lo + s) * kStage;
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(m),
                   "r"((uint32_t)(kCodes + (kBf16 ? kBTile : 0)))
                   : "memory");
      copy2d(sb + (t & 3) * kCodes, &tm_w, k0 / 2, n0, m);
      if (kBf16)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          copy2d(sb + kX0 + (t & 3) * kBTile + h * (kBTile / 2), &tm_x, k0 + 64 * h, r0, m);
    };
    // Scales and fp32 rows of x of two stages in registers, ahead of use.
    __half sn[2];
    float xv[2][kBf16 ? 1 : kParts][8];
    auto fetch = [&](int u, int s) {
      // (a group behind the last one counts as 0 against any scale)
      if (piece < kGroups) {
        const int g = (s_lo + s) * kGroups + piece;
        sn[u] = g < groups ? __ldg(sp + g) : __half(0.f);
      }
      if constexpr (!kBf16) {
        const int k = (s_lo + s) * kStage + 8 * (tid & 15);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const int r = (tid + i * kThreads) >> 4;
          const bool on = r < nr && k < P.K;
          const float4 *p = reinterpret_cast<const float4 *>(
              static_cast<const float *>(P.x) + (on ? (size_t)(r0 + r) * P.K + k : 0));
          const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 a = on ? __ldg(p) : z, b = on ? __ldg(p + 1) : z;
          const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) xv[u][i][j] = v[j];
        }
      }
    };
    if (tid == 0)
      for (int s = 0; s < min(ns, kRing); ++s) copy(s);
    if (ns > 0) fetch(0, 0);
    if (ns > 1) fetch(1, 1);
    for (int s0 = 0; s0 < ns + kLag; s0 += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int s = s0 + u;
        const uint32_t at = base + (uint32_t)s, before = at - kLag;  // over all passes
        if (s >= kLag && s < ns + kLag) {
          // stage s - kLag: its buffers are free, its accumulators full
          failed |= !mbar_wait(bar + 8 * (before & 1), (before >> 1) & 1u, kWaitLimit);
          if (tid == 0 && s - kLag + kRing < ns) copy(s - kLag + kRing);
          fence_after_sync();
          constexpr int kAt = kGroups * kCols > 32 ? 32 / kCols : kGroups;  // groups at a time
#pragma unroll
          for (int g0 = 0; g0 < kGroups; g0 += kAt) {
            uint32_t d[kAt][kCols];
#pragma unroll
            for (int g = 0; g < kAt; ++g)
              tmem_ld_async(
                  tl + (uint32_t)(((before % kLag) * kGroups + g0 + g) * kNC + part * kCols), d[g]);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int g = 0; g < kAt; ++g) {
              const float f = scl[((before & 3) * 4 + g0 + g) * kRowsW + row];
#pragma unroll
              for (int i = 0; i < kCols; ++i) {
                asm volatile("" : "+r"(d[g][i]));  // defined only from the wait on
                acc[i] = fmaf(f, __uint_as_float(d[g][i]), acc[i]);
              }
            }
          }
        }
        if (s >= ns) continue;
        if (piece < kGroups) scl[((at & 3) * 4 + piece) * kRowsW + srow] = __half2float(sn[u]);
        failed |= !mbar_wait(full + 8 * (at & 3), (at >> 2) & 1u, kWaitLimit);
        {
          const uint4 w = *reinterpret_cast<const uint4 *>(wp + (at & 3) * kCodes);
          const uint32_t word[4] = {w.x, w.y, w.z, w.w};
          const uint32_t a = tl + kAcc + (at & 1) * 64 + 16 * part;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[8];
            codes(word[2 * h], r);
            codes(word[2 * h + 1], r + 4);
            tmem_st8_async(a + 8 * h, r);
          }
        }
        if constexpr (!kBf16) {
          unsigned char *B = gb + kX0 + (at & 1) * 3 * kBTile;
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            const int e = tid + i * kThreads;
            unsigned char *dst = B + sw128_off(kNC, e >> 4, 8 * (e & 15), 2);
            float(&x)[8] = xv[u][i];
#pragma unroll
            for (int term = 0; term < 3; ++term, dst += kBTile) {
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                // (cut off, so no finite element becomes infinite; the third
                // part is exact: 3 x 8 bits)
                const uint32_t p = __float_as_uint(x[2 * j]), q = __float_as_uint(x[2 * j + 1]);
                o[j] = __byte_perm(p, q, 0x7632);
                x[2 * j] -= __uint_as_float(p & 0xffff0000u);
                x[2 * j + 1] -= __uint_as_float(q & 0xffff0000u);
              }
              *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        if (s + 2 < ns) fetch(u, s + 2);
        tmem_wait_st();
        if (!kBf16) fence_proxy_async();
        fence_before_sync();
        __syncthreads();
        if (warp == 0) {
          fence_after_sync();
          const uint32_t one = elect();
          const uint32_t a = tmem + kAcc + (at & 1) * 64;
          const uint32_t b = sb + kX0 + (kBf16 ? (at & 3) * kBTile : (at & 1) * 3 * kBTile);
          constexpr uint32_t id = idesc(kFmtBF16, kRowsW, kNC);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const uint32_t d = tmem + (uint32_t)(((at % kLag) * kGroups + g) * kNC);
#pragma unroll
            for (int term = kTerms - 1; term >= 0; --term)  // (small ones first)
#pragma unroll
              for (int k = 0; k < kGroup / 16; ++k) {
                const int ks = g * (kGroup / 16) + k;
                mma_ts(one, d, a + 8u * ks, desc_kstep(b + term * kBTile, kNC, ks), id,
                       term < kTerms - 1 || k > 0);
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
    const int n = n0 + row;
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

// rows x cols elements, boxes of box_rows x box_cols; zeros outside.
bool map2d(CUtensorMap *map, CUtensorMapDataType type, const void *base, int cols, int rows,
           int bytes, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * bytes};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return fn != nullptr &&
         fn(map, type, 2, const_cast<void *>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kBf16, int kNC, int kGroup>
cudaError_t launch(const WideArgs &a, int tiles, cudaStream_t stream) {
  const auto kernel = quant_wide_kernel<kBf16, kNC, kGroup>;
  constexpr int bytes = smem_bytes<kBf16, kNC>();
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  CUtensorMap w, x = {};
  if (!map2d(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.qw, a.K / 2, a.N, 1, 64, kRowsW,
             CU_TENSOR_MAP_SWIZZLE_64B) ||
      (kBf16 && !map2d(&x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.rows, 2, 64, kNC,
                       CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
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
  return cudaLaunchKernelEx(&cfg, kernel, w, x, a);
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
