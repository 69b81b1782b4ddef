// Linear layers of few rows on tcgen05 tensor cores, forward and the input's gradient:
//   out[t, n] = act(sum_k x[t, k] w[n, k] + bias[n]) + residual[t, n]
//   g_x[t, k] = sum_n g_p[t, n] w[n, k]
//
// With few rows the weights' bytes bound the product (one row of 4096 -> 16384:
// 134 MB, 20 us of HBM time), so the weights are the MMA's A operand - 128 features are
// the TMEM lanes - and the rows its N: no lane is wasted on rows that are not there, and
// one row costs the tensor cores as little as 16.  In the gradient the contracted index
// is the slow one of w, which tcgen05 takes as an MN-major A tile.
//
// A cluster of C CTAs shares a tile of 128 features, each a range of the contracted
// index, so that few tiles still fill the GPU; their float32 tiles meet in shared memory
// (no round trip through global memory, no second kernel): each CTA writes to the others
// what they finish and adds what it got in rank order, so two runs give the same bits.
// (Left for the others to read: 8 x 4096 -> 1024 6.6 us instead of 5.3.)
#include <cuda.h>

#include "block_epilogue.cuh"
#include "jmix_internal.cuh"
#include "sm100.cuh"

namespace jmix {
namespace {

using namespace sm100;

constexpr int kThreads = 192;          // weights' and rows' producer, MMA, 4 drain warps
constexpr int kK = 64;                 // K chunk: one 128-byte swizzle span
constexpr int kTile = 128;             // features of a tile
constexpr int kWBytes = kTile * kK * 2;
constexpr int kMaxStages = 12;
constexpr int kMaxCluster = 8;
constexpr size_t kSmemSm = 227 * 1024;

struct FewArgs {
  int T, nb;             // rows; rounded up to the MMA's N
  int chunks, stages;
  unsigned tmem_cols;
  int64_t N;             // features of the output
  Epilogue ep;
  ErrFlags* err;
  bool clear_err;
  bool late_wait;   // wait for the kernel before this one at the end
};

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}

// AMN: w is stored [contracted][features], else [features][contracted].
template <bool AMN>
__global__ void __launch_bounds__(kThreads)
    k_linear_few(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                 const FewArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t tmem_slot;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = g.stages, stage_bytes = kWBytes + g.nb * 128;
  const uint32_t rank = cluster_rank(), C = cluster_size();
  const int64_t n0 = (int64_t)(blockIdx.x / C) * kTile;
  const int k0 = (int)((unsigned)g.chunks * rank / C), k1 = (int)((unsigned)g.chunks * (rank + 1) / C);

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(&done), 1);
    fence_mbar_init();
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), g.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot, base = smem_u32(smem);
  if (!g.late_wait) {
    // The ring's first weights on their way to L2 while the kernel before ends (L2 sees what
    // that one still writes; shared memory would not).  1 x 4096 -> 16384: 24.4 -> 22.4 us,
    // 16 x 14336 -> 4096 22.3 -> 20.6; twice the ring's is slower between other kernels (norm,
    // 1 x 4096 -> 16384, back: 48.5 -> 51.5 us), and k_linear_pair gains nothing by it.
    if (warp == 0 && elect_one())
      for (int kc = k0; kc < k1 && kc < k0 + S; ++kc) {
        if constexpr (AMN) {
          tma_prefetch_3d(&tm_w, (int32_t)n0, kc * kK, 0);
          tma_prefetch_3d(&tm_w, (int32_t)n0 + 64, kc * kK, 0);
        } else {
          tma_prefetch_3d(&tm_w, kc * kK, (int32_t)n0, 0);
        }
      }
    grid_dep_wait();
  }
  grid_dep_launch();
  // (a wait gives up after 2 s: no CTA can have recorded one yet)
  if (g.clear_err && blockIdx.x == 0 && tid < (int)(sizeof(ErrFlags) / 4))
    reinterpret_cast<unsigned*>(g.err)[tid] = 0u;

  if (warp == 0) {
    if (elect_one()) {
      const uint64_t pol = l2_evict_first_policy();   // weights pass through once
      int s = 0;
      uint32_t parity = 1;   // the first round's wait for "empty" returns at once
      for (int kc = k0; kc < k1; ++kc) {
        if (!mbar_wait(smem_u32(&empty[s]), parity, g.err, 101)) break;
        const uint32_t fb = smem_u32(&full[s]), dst = base + (uint32_t)(s * stage_bytes);
        mbar_arrive_expect_tx(fb, (uint32_t)stage_bytes);
        if constexpr (AMN) {   // boxes of 64 features x 64 contracted rows
          tma_load_3d(dst, &tm_w, fb, (int32_t)n0, kc * kK, 0, pol);
          tma_load_3d(dst + kWBytes / 2, &tm_w, fb, (int32_t)n0 + 64, kc * kK, 0, pol);
        } else {
          tma_load_3d(dst, &tm_w, fb, kc * kK, (int32_t)n0, 0, pol);
        }
        tma_load_2d(dst + kWBytes, &tm_x, fb, kc * kK, 0);
        if (++s == S) {
          s = 0;
          parity ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16_f32_major(kTile, g.nb, AMN, false);
      int s = 0;
      uint32_t parity = 0;
      bool ok = true;
      for (int kc = k0; kc < k1; ++kc) {
        if (!mbar_wait(smem_u32(&full[s]), parity, g.err, 102)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t wa = base + (uint32_t)(s * stage_bytes), xb = wa + kWBytes;
#pragma unroll
        for (int kk = 0; kk < kK / 16; ++kk)
          umma_f16(tmem,
                   AMN ? sw128_mnmajor_desc(wa + kk * 2048, kWBytes / 2)
                       : sw128_kmajor_desc(wa + kk * 32),
                   sw128_kmajor_desc(xb + kk * 32), idesc, (kc > k0 || kk > 0) ? 1u : 0u);
        umma_commit(smem_u32(&empty[s]));
        if (++s == S) {
          s = 0;
          parity ^= 1u;
        }
      }
      if (ok) umma_commit(smem_u32(&done));
    }
  }
  // CTA q of the cluster finishes F features of all rows; the others write theirs of them,
  // float32, to its shared memory, [CTA][row][feature], in the ring's place: once the MMAs of
  // all have consumed their rings.
  const int F = kTile / (int)C;
  if (warp >= 2) {
    const int lg = warp & 3, et = lg * 32 + lane;   // TMEM lane = feature of the tile
    const bool ok = mbar_wait(smem_u32(&done), 0, g.err, 103);
    __syncwarp();
    cluster_arrive();
    tc_fence_after();
    const uint32_t tb = tmem + ((uint32_t)(lg * 32) << 16);
    const uint32_t to = cluster_addr(base, (uint32_t)(et / F)) +
                        ((uint32_t)((int)rank * g.nb * F) + (uint32_t)(et % F)) * 4;
    for (int c = 0; c < g.nb; c += 16) {
      uint32_t r[16];
      tmem_ld16(tb + (uint32_t)c, r);
      tmem_ld_wait();
      if (c == 0) cluster_wait();
      if (ok) {
#pragma unroll
        for (int i = 0; i < 16; ++i) st_cluster(to + (uint32_t)((c + i) * F) * 4, r[i]);
      }
    }
  } else {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_before();
  cluster_sync();
  // in rank order, 8 features of a row at a time
  const float* parts = reinterpret_cast<const float*>(smem);
  const int f8 = F / 8, items = g.T * f8;
  for (int i = tid; i < items; i += kThreads) {
    const int t = i / f8, f = (i - t * f8) * 8;
    const int64_t col = n0 + rank * F + f;
    if (col >= g.N) continue;
    const float* p = parts + t * F + f;
    float v[8] = {};
#pragma unroll 4
    for (uint32_t q = 0; q < C; ++q, p += g.nb * F) {
      const float4 a = *reinterpret_cast<const float4*>(p);
      const float4 b = *reinterpret_cast<const float4*>(p + 4);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    finish8(g.ep, v, (int64_t)t * g.N + col, col);
  }
  if (g.late_wait) grid_dep_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, g.tmem_cols);
  }
}

// ------------------------------------------------------------------ host side

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool map(CUtensorMap* m, const void* base, int64_t rows, int64_t inner, int box, int rank) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, 1};
  cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)(inner * rows) * 2};
  cuuint32_t bx[3] = {kK, (cuuint32_t)box, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims,
            strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How the product is cut: CTAs of a cluster, ring stages and shared memory of one.
struct FewShape {
  int nb, cluster, stages;
  size_t smem;
};

// The least estimated time over cluster sizes and one or two CTAs an SM (two hide each
// other's start and end and let up to 296 CTAs stream at once, with rings of half the
// size).  What passes through an SM, rows included, goes at 0.095 MB/us at most; the stream
// from HBM at 6.9 MB/us with 1.8 MB on their way at least, and slower with few SMs at it; a
// wave of CTAs starts and ends in 3.2 us; what a cluster's CTAs write to each other grows with
// the rows and the CTAs.  Measured, us: 16 x 8192 -> 8192 with clusters of 1, 2 and 4 CTAs,
// one an SM, 28.1, 22.9, 25.6 (two rounds), two an SM 31.8, 25.9, 21.7; 1 x 1024 -> 1024 6.3,
// 4.9, 4.2 and of 8 CTAs 3.8; 100 x 4096 -> 4096 18.6, 12.6, 10.7, 22.7 (three rounds).
FewShape few_shape(int64_t T, int64_t N, int64_t K) {
  // clusters of 1, 2, 4 and 8 CTAs that a B200 holds, with one or two CTAs an SM
  static const int kClusters[2][9] = {{0, 148, 74, 0, 33, 0, 0, 0, 15},
                                      {0, 296, 148, 0, 71, 0, 0, 0, 33}};
  FewShape f{};
  f.nb = (int)(ceil_div(T, 16) * 16);
  const int64_t tiles = ceil_div(N, kTile), chunks = ceil_div(K, kK);
  const size_t stage = kWBytes + (size_t)f.nb * 128, tile = (size_t)f.nb * kTile * 4;
  const double hbm = (double)N * (double)K * 2.0 / 6.9e6;
  double best = 1e30;
  for (int c = 1; c <= kMaxCluster; c *= 2) {
    if (c > 1 && chunks / c < 2) break;
    const int64_t ctas = tiles * c, steps = ceil_div(chunks, c);
    for (int per = 1; per <= 2; ++per) {
      const size_t most = kSmemSm / per - 3072;
      int64_t stages = (int64_t)(most / stage);
      if (stages < 3 || tile > most) break;
      if (stages > kMaxStages) stages = kMaxStages;
      if (stages > steps) stages = steps;
      const int64_t held = kClusters[per - 1][c], waves = ceil_div(tiles, held);
      const int64_t at_once = ctas < held * c ? ctas : held * c;
      const int64_t on_sm = ctas < 148 * per ? ceil_div(ctas, 148) : per;
      const double through = (double)(waves * on_sm * steps) * (double)stage / 0.095e6;
      double us = hbm * (1.0 + 1.8e6 / ((double)(at_once * stages) * (double)kWBytes));
      if (at_once < 148) us *= 1.2 - 0.2 * (double)at_once / 148.0;
      if (us < through) us = through;
      us += 3.2 * (double)waves;
      if (c > 1) us += (double)c * (0.02 + 0.0055 * (double)(f.nb - 16));
      if (us < best * 0.995) {
        best = us;
        f.cluster = c;
        f.stages = (int)stages;
        const size_t ring = f.stages * stage;
        f.smem = 1024 + (ring > tile ? ring : tile);
      }
    }
  }
  return f;
}

template <bool AMN>
cudaError_t launch_few(const CUtensorMap& w, const CUtensorMap& x, const FewArgs& g,
                       const FewShape& f, int64_t tiles, cudaStream_t s) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(k_linear_few<AMN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kSmemSm - 2048));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * f.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = f.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)f.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_linear_few<AMN>, w, x, g);
}

}  // namespace

// Up to 64 rows, and up to 192 over a long contracted index, whatever the number of features
// (measured with 1024 to 8192): a tile's exchange grows with the rows, k_linear_pair's does not,
// but its 256-row tiles read the weights no faster for few rows.  Microseconds here and there: 96 rows, 512 -> 4096 6.2, 5.5; 1024 -> 4096 7.0, 7.2;
// 128 rows, 1024 -> 1024 6.6, 6.2; 8192 -> 4096 15.8, 19.2; 160 rows, 2048 -> 4096 9.3, 8.9;
// 4096 -> 8192 17.5, 20.1; 192 rows, 4096 -> 1024 10.4, 9.1; 8192 -> 4096 18.5, 19.6; 256
// rows, 8192 -> 4096 21.9, 19.8.
bool linear_few(int64_t rows, int64_t contracted) {
  const int64_t most = contracted <= 1024   ? 64
                       : contracted < 4096 ? 128
                       : contracted < 8192 ? 160
                                           : 192;
  return rows <= most;
}

cudaError_t run_linear_few(int64_t T, int64_t N, int64_t K, const void* x, const void* w, bool w_mn,
                           const Epilogue& ep, ErrFlags* err, bool clear_err, bool apart, Problem& p) {
  const FewShape f = few_shape(T, N, K);
  FewArgs g{};
  g.T = (int)T;
  g.nb = f.nb;
  g.chunks = (int)ceil_div(K, kK);
  g.stages = f.stages;
  g.tmem_cols = 32;
  while (g.tmem_cols < (unsigned)f.nb) g.tmem_cols *= 2;
  g.N = N;
  g.ep = ep;
  g.err = err;
  g.clear_err = clear_err;
  g.late_wait = apart && !clear_err;
  CUtensorMap tw, tx;
  if (!(w_mn ? map(&tw, w, K, N, 64, 3) : map(&tw, w, N, K, kTile, 3)) ||
      !map(&tx, x, T, K, f.nb, 2))
    return cudaErrorInvalidValue;
  const int64_t tiles = ceil_div(N, kTile);
  const cudaError_t e = w_mn ? launch_few<true>(tw, tx, g, f, tiles, p.stream)
                             : launch_few<false>(tw, tx, g, f, tiles, p.stream);
  if (e == cudaSuccess) launched(p, "k_linear_few");
  return e;
}

}  // namespace jmix
