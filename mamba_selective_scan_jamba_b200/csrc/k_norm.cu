// LayerNorm / RMSNorm over the rows of a matrix, with the residual add before
// it, and its backward with the weight's and bias's gradients.
//
//   s    = x + r, rounded to the io type (the value the residual stream carries)
//   y    = (s - m) rstd w + b,  rstd = (mean((s - m)^2) + eps)^-1/2,
//          m = mean(s) (LayerNorm) or 0 (RMSNorm)
//   xh   = (s - m) rstd,  g = gy w
//   g_x  = rstd (g - [mean(g)] - xh mean(g xh)) + g_sum
//   g_w  = sum over rows of gy xh,  g_b = sum over rows of gy
//
// Both passes are bound by HBM: a row is read once into registers and every
// statistic is taken from there, so the forward moves 2 (4 with a residual) and
// the backward 3 (4) values per element.  The variance is the mean of the squared
// differences from the mean (two reductions over registers), not E[s^2] - m^2,
// which cancels for rows far from zero.  All arithmetic is float32; y, sum and
// the gradients are rounded once to the io type.
//
// A group of `wpr` warps owns a row; a thread keeps NV vectors of VEC values
// (16-byte accesses, or 8, 4 or 2 where the width or the stride of x asks for them).  In the backward a group walks over rows with a stride, so that each
// thread owns its columns of g_w and g_b and sums them in registers; the groups'
// partial rows go to the workspace and k_norm_bwd_reduce adds them in a fixed
// order (the same bits on every run).  k_norm_bwd_ring has the rows of g_y, x and g_sum
// copied into a ring in shared memory some rows ahead (with loads of the next row only,
// 8192 x 4096 bf16 with g_sum took 109 us, with the ring 51 us); k_norm_bwd loads them
// itself, for rows of x that lie apart by no multiple of 16 bytes and rows that no ring has
// room for.
#include "jmix_internal.cuh"
#include "sm100.cuh"

namespace jmix {
namespace {

using sm100::grid_dep_launch;
using sm100::grid_dep_wait;

constexpr int kNormSMs = 148;
constexpr int kNormMaxStages = 6;

// VEC values as one access: 16, 8 or 4 bytes, or a single value.
template <typename T, int VEC, int BYTES>
struct RawOf {
  using type = T;
};
template <typename T, int VEC>
struct RawOf<T, VEC, 16> {
  using type = uint4;
};
template <typename T, int VEC>
struct RawOf<T, VEC, 8> {
  using type = uint2;
};
template <>
struct RawOf<__nv_bfloat16, 2, 4> {
  using type = uint32_t;
};
template <typename T, int VEC>
using Raw = typename RawOf<T, VEC, VEC * sizeof(T)>::type;

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Raw<T, VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = static_cast<float>(r);
  } else {
    constexpr int W = VEC * sizeof(T) / 4;
    uint32_t u[W];
    if constexpr (W == 1) {
      u[0] = r;
    } else {
      u[0] = r.x;
      u[1] = r.y;
      if constexpr (W == 4) {
        u[2] = r.z;
        u[3] = r.w;
      }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(u[i]);
      } else {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> pack(const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    return static_cast<T>(f[0]);
  } else {
    constexpr int W = VEC * sizeof(T) / 4;
    uint32_t u[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(T) == 4) {
        u[i] = __float_as_uint(f[i]);
      } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    if constexpr (W == 1)
      return u[0];
    else if constexpr (W == 2)
      return make_uint2(u[0], u[1]);
    else
      return make_uint4(u[0], u[1], u[2], u[3]);
  }
}

template <typename R>
__device__ __forceinline__ R zero_raw() {
  if constexpr (sizeof(R) == 16)
    return make_uint4(0u, 0u, 0u, 0u);
  else if constexpr (sizeof(R) == 8)
    return make_uint2(0u, 0u);
  else
    return R{};
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over the group's threads (every thread of the CTA calls it together;
// `red` holds one value per warp of the CTA and is not reused before the next
// barrier of the caller).
__device__ __forceinline__ float group_sum(float v, float* red, int wpr) {
  v = warp_sum(v);
  if (wpr == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int first = warp / wpr * wpr;
  return warp_sum(lane < wpr ? red[first + lane] : 0.0f);
}

template <typename T, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) k_norm_fwd(const NormFwdArgs a) {
  __shared__ float red[2][32];
  using R = Raw<T, VEC>;
  const int gthreads = 32 * a.wpr;
  const int group = threadIdx.x / gthreads, t = threadIdx.x - group * gthreads;
  const int64_t row = (int64_t)blockIdx.x * a.rpc + group;
  const bool live = row < a.rows;
  const int nvec = (int)(a.cols / VEC);
  grid_dep_wait();
  grid_dep_launch();
  const R* x = reinterpret_cast<const R*>(static_cast<const T*>(a.x) + (live ? row : 0) * a.x_stride);
  const int64_t base = (live ? row : 0) * (int64_t)nvec;
  const R* res = a.residual ? static_cast<const R*>(a.residual) + base : nullptr;
  const R* wp = static_cast<const R*>(a.weight);
  const R* bp = static_cast<const R*>(a.bias);
  R rx[NV], rr[NV], rw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * gthreads + t;
    const bool ok = live && i < nvec;
    rx[v] = ok ? x[i] : zero_raw<R>();
    if (res) rr[v] = ok ? res[i] : zero_raw<R>();
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * gthreads + t;
    rw[v] = i < nvec ? wp[i] : zero_raw<R>();
  }
  float s[NV][VEC];
  float acc = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    unpack<T, VEC>(rx[v], s[v]);
    if (res) {
      float q[VEC];
      unpack<T, VEC>(rr[v], q);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[v][j] += q[j];
      // the normalised value is the stored one, so that the backward, which
      // reads `sum`, differentiates what was computed here
      const R p = pack<T, VEC>(s[v]);
      unpack<T, VEC>(p, s[v]);
      const int i = v * gthreads + t;
      if (live && i < nvec) (static_cast<R*>(a.sum) + base)[i] = p;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc += a.layer ? s[v][j] : s[v][j] * s[v][j];
  }
  const float inv_n = 1.0f / (float)a.cols;
  float mean = 0.0f, var;
  if (a.layer) {
    mean = group_sum(acc, red[0], a.wpr) * inv_n;
    acc = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v * gthreads + t < nvec)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc = fmaf(s[v][j] - mean, s[v][j] - mean, acc);
    var = group_sum(acc, red[1], a.wpr) * inv_n;
  } else {
    var = group_sum(acc, red[0], a.wpr) * inv_n;
  }
  const float rstd = 1.0f / sqrtf(var + a.eps);
  if (!live) return;
  R* y = static_cast<R*>(a.y) + base;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * gthreads + t;
    if (i >= nvec) break;
    float w[VEC], o[VEC];
    unpack<T, VEC>(rw[v], w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = (s[v][j] - mean) * rstd * w[j];
    if (bp) {
      float b[VEC];
      unpack<T, VEC>(bp[i], b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] += b[j];
    }
    y[i] = pack<T, VEC>(o);
  }
  if (a.stats && t == 0) {
    a.stats[2 * row] = mean;
    a.stats[2 * row + 1] = rstd;
  }
}

template <typename T, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1) k_norm_bwd(const NormBwdArgs a) {
  __shared__ float red[2][2][32];
  using R = Raw<T, VEC>;
  const int gthreads = 32 * a.wpr;
  const int group = threadIdx.x / gthreads, t = threadIdx.x - group * gthreads;
  const int nvec = (int)(a.cols / VEC);
  const int64_t step = (int64_t)gridDim.x * a.rpc;
  const int64_t first = (int64_t)blockIdx.x * a.rpc + group;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x < sizeof(ErrFlags) / 4)
    reinterpret_cast<unsigned*>(a.err)[threadIdx.x] = 0u;
  const R* wp = static_cast<const R*>(a.weight);
  R rw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * gthreads + t;
    rw[v] = i < nvec ? wp[i] : zero_raw<R>();
  }
  float gw[NV][VEC], gb[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < VEC; ++j) gw[v][j] = gb[v][j] = 0.0f;
  const float inv_n = 1.0f / (float)a.cols;

  R rx[NV], rg[NV];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t row) {
    const bool live = row < a.rows;
    const R* x = reinterpret_cast<const R*>(static_cast<const T*>(a.x) + (live ? row : 0) * a.x_stride);
    const R* g = static_cast<const R*>(a.gy) + (live ? row : 0) * (int64_t)nvec;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * gthreads + t;
      const bool ok = live && i < nvec;
      rx[v] = ok ? x[i] : zero_raw<R>();
      rg[v] = ok ? g[i] : zero_raw<R>();
    }
    mean = live ? a.stats[2 * row] : 0.0f;
    rstd = live ? a.stats[2 * row + 1] : 0.0f;
  };
  load(first);
  // every group of the CTA runs the same number of rounds (barriers inside)
  const int64_t rounds = (a.rows - (int64_t)blockIdx.x * a.rpc + step - 1) / step;
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t row = first + it * step;
    const bool live = row < a.rows;
    const int64_t base = (live ? row : 0) * (int64_t)nvec;
    float xh[NV][VEC], g[NV][VEC];
    float sg = 0.0f, sgx = 0.0f;
    const float rs = rstd;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w[VEC];
      unpack<T, VEC>(rx[v], xh[v]);
      unpack<T, VEC>(rg[v], g[v]);
      unpack<T, VEC>(rw[v], w);
      const bool in = live && v * gthreads + t < nvec;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        xh[v][j] = in ? (xh[v][j] - mean) * rs : 0.0f;
        gw[v][j] = fmaf(g[v][j], xh[v][j], gw[v][j]);
        gb[v][j] += g[v][j];
        g[v][j] *= w[j];
        sg += g[v][j];
        sgx = fmaf(g[v][j], xh[v][j], sgx);
      }
    }
    load(row + step);  // in flight during this row's reductions
    sg = warp_sum(sg);
    sgx = warp_sum(sgx);
    if (a.wpr > 1) {
      float(*rd)[32] = red[it & 1];
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      if (lane == 0) {
        rd[0][warp] = sg;
        rd[1][warp] = sgx;
      }
      __syncthreads();
      const int w0 = warp / a.wpr * a.wpr;
      sg = warp_sum(lane < a.wpr ? rd[0][w0 + lane] : 0.0f);
      sgx = warp_sum(lane < a.wpr ? rd[1][w0 + lane] : 0.0f);
    }
    const float c0 = a.layer ? sg * inv_n : 0.0f, c1 = sgx * inv_n;
    if (live) {
      const R* gs = a.g_sum ? static_cast<const R*>(a.g_sum) + base : nullptr;
      R* gx = static_cast<R*>(a.g_x) + base;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = v * gthreads + t;
        if (i >= nvec) break;
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = (g[v][j] - c0 - xh[v][j] * c1) * rs;
        if (gs) {
          float q[VEC];
          unpack<T, VEC>(gs[i], q);
#pragma unroll
          for (int j = 0; j < VEC; ++j) o[j] += q[j];
        }
        gx[i] = pack<T, VEC>(o);
      }
    }
  }
  if (a.part) {
    float* pw = a.part + ((int64_t)blockIdx.x * a.rpc + group) * 2 * a.cols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * gthreads + t;
      if (i >= nvec) break;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        pw[(int64_t)i * VEC + j] = gw[v][j];
        pw[a.cols + (int64_t)i * VEC + j] = gb[v][j];
      }
    }
  }
}

// Shared memory of one array's rows in a stage of the backward's ring.
__host__ __device__ inline uint32_t ring_part_bytes(size_t rows_bytes, bool ragged) {
  return (uint32_t)(ragged ? (rows_bytes + 15) / 16 * 16 + 16 : rows_bytes);
}

// The backward with its rows copied ahead.  A round takes the CTA's next rpc rows; the
// stage they came from is refilled for the round `stages` later at the round's barrier,
// when every thread holds its values in registers.
template <typename T, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) k_norm_bwd_ring(const NormBwdArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][2][32];
  __shared__ uint64_t full[kNormMaxStages];
  using R = Raw<T, VEC>;
  constexpr bool kRagged = VEC * sizeof(T) < 16;
  const int gthreads = 32 * a.wpr;
  const int group = threadIdx.x / gthreads, t = threadIdx.x - group * gthreads;
  const int nvec = (int)(a.cols / VEC), S = a.stages;
  const uint32_t row_bytes = (uint32_t)(a.cols * sizeof(T));
  const uint32_t part_bytes = ring_part_bytes(a.rpc * (size_t)row_bytes, kRagged);
  const uint32_t stage_bytes = part_bytes * (a.g_sum ? 3 : 2);
  // Rows that are no multiple of 16 bytes come with what is around them up to the
  // next 16-byte boundaries; behind `safe` they would end outside the tensor.
  const int64_t safe = a.rows * row_bytes & ~int64_t(15);
  const int64_t step = (int64_t)gridDim.x * a.rpc, first = (int64_t)blockIdx.x * a.rpc;
  const int64_t rounds = (a.rows - first + step - 1) / step;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) sm100::mbar_init(sm100::smem_u32(&full[i]), 1);
    sm100::fence_mbar_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x < sizeof(ErrFlags) / 4)
    reinterpret_cast<unsigned*>(a.err)[threadIdx.x] = 0u;
  auto fill = [&](int64_t it, int s) {   // one thread
    const int64_t row = first + it * step, left = a.rows - row;
    const uint32_t n = left < a.rpc ? (uint32_t)left : (uint32_t)a.rpc;
    const uint32_t bar = sm100::smem_u32(&full[s]);
    uint32_t dst = sm100::smem_u32(ring) + s * stage_bytes;
    if constexpr (kRagged) {
      const int64_t r0 = row * row_bytes & ~int64_t(15);
      const int64_t r1 = min((row + n) * row_bytes + 15 & ~int64_t(15), safe);
      const uint32_t bytes = r1 > r0 ? (uint32_t)(r1 - r0) : 0u;
      sm100::mbar_arrive_expect_tx(bar, bytes * (a.g_sum ? 3 : 2));
      if (bytes == 0) return;
      sm100::bulk_load(dst, static_cast<const char*>(a.x) + r0, bytes, bar);
      sm100::bulk_load(dst + part_bytes, static_cast<const char*>(a.gy) + r0, bytes, bar);
      if (a.g_sum)
        sm100::bulk_load(dst + 2 * part_bytes, static_cast<const char*>(a.g_sum) + r0, bytes, bar);
      return;
    }
    sm100::mbar_arrive_expect_tx(bar, n * row_bytes * (a.g_sum ? 3 : 2));
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    if (a.x_stride == a.cols)
      sm100::bulk_load(dst, x, n * row_bytes, bar);
    else
      for (uint32_t i = 0; i < n; ++i)
        sm100::bulk_load(dst + i * row_bytes, x + i * a.x_stride, row_bytes, bar);
    sm100::bulk_load(dst + part_bytes, static_cast<const T*>(a.gy) + row * a.cols, n * row_bytes,
                     bar);
    if (a.g_sum)
      sm100::bulk_load(dst + 2 * part_bytes, static_cast<const T*>(a.g_sum) + row * a.cols,
                       n * row_bytes, bar);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < S && i < rounds; ++i) fill(i, i);
  const R* wp = static_cast<const R*>(a.weight);
  R rw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * gthreads + t;
    rw[v] = i < nvec ? wp[i] : zero_raw<R>();
  }
  float gw[NV][VEC], gb[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < VEC; ++j) gw[v][j] = gb[v][j] = 0.0f;
  const float inv_n = 1.0f / (float)a.cols;
  const float2* stats = reinterpret_cast<const float2*>(a.stats);
  float2 st = first + group < a.rows ? stats[first + group] : make_float2(0.0f, 0.0f);
  int s = 0;
  uint32_t parity = 0;
  bool ok = true;
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t row = first + it * step + group;
    const bool live = row < a.rows;
    // (a group without a row adds zeros whatever its last row's statistics were)
    const float mean = live ? st.x : 0.0f, rs = live ? st.y : 0.0f;
    if (row + step < a.rows) st = stats[row + step];
    ok = ok && sm100::mbar_wait(sm100::smem_u32(&full[s]), parity, a.err, 111);
    uint8_t* stage = ring + s * stage_bytes;
    uint32_t at = (uint32_t)group * row_bytes;
    if constexpr (kRagged) {
      const int64_t r0 = first + it * step, from = r0 * row_bytes & ~int64_t(15);
      at = (uint32_t)(row * row_bytes - from);
      if (r0 + a.rpc >= a.rows && safe < a.rows * row_bytes) {   // (uniform in the CTA)
        // the values behind `safe`, at most 7 of each array
        const int n = (int)((a.rows * row_bytes - safe) / sizeof(T)), q = threadIdx.x;
        if (q < n * (a.g_sum ? 3 : 2)) {
          const int k = q / n;
          const void* array = k == 0 ? a.x : k == 1 ? a.gy : a.g_sum;
          reinterpret_cast<T*>(stage + k * part_bytes + (safe - from))[q - k * n] =
              reinterpret_cast<const T*>(static_cast<const char*>(array) + safe)[q - k * n];
        }
        __syncthreads();
      }
    }
    const R* sx = reinterpret_cast<const R*>(stage + at);
    const R* sgy = reinterpret_cast<const R*>(stage + part_bytes + at);
    const R* ssum = reinterpret_cast<const R*>(stage + 2 * part_bytes + at);
    float xh[NV][VEC], g[NV][VEC];
    R rs_sum[NV];
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * gthreads + t;
      const bool in = live && i < nvec;
      const R rx = in ? sx[i] : zero_raw<R>();
      const R rg = in ? sgy[i] : zero_raw<R>();
      rs_sum[v] = in && a.g_sum ? ssum[i] : zero_raw<R>();
      float w[VEC];
      unpack<T, VEC>(rx, xh[v]);
      unpack<T, VEC>(rg, g[v]);
      unpack<T, VEC>(rw[v], w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        xh[v][j] = (xh[v][j] - mean) * rs;   // (behind the row's end g is 0)
        gw[v][j] = fmaf(g[v][j], xh[v][j], gw[v][j]);
        gb[v][j] += g[v][j];
        g[v][j] *= w[j];
        sg += g[v][j];
        sgx = fmaf(g[v][j], xh[v][j], sgx);
      }
    }
    // both sums in one tree: after the first exchange the lower lanes carry sg, the upper sgx
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool upper = lane >= 16;
    float both = (upper ? sgx : sg) + __shfl_xor_sync(0xffffffffu, upper ? sg : sgx, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) both += __shfl_xor_sync(0xffffffffu, both, o);
    float(*rd)[32] = red[it & 1];
    if (a.wpr > 1 && (lane & 15) == 0) rd[lane >> 4][warp] = both;
    __syncthreads();
    if (threadIdx.x == 0 && ok && it + S < rounds) fill(it + S, s);
    if (++s == S) {
      s = 0;
      parity ^= 1u;
    }
    if (a.wpr > 1) {
      const int w0 = warp / a.wpr * a.wpr, q = lane & 15;
      both = q < a.wpr ? rd[lane >> 4][w0 + q] : 0.0f;
      if (a.wpr > 16 && q + 16 < a.wpr) both += rd[lane >> 4][w0 + q + 16];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) both += __shfl_xor_sync(0xffffffffu, both, o);
    }
    const float other = __shfl_xor_sync(0xffffffffu, both, 16);
    sg = upper ? other : both;
    sgx = upper ? both : other;
    const float c0 = a.layer ? sg * inv_n : 0.0f, c1 = sgx * inv_n;
    if (live) {
      R* gx = static_cast<R*>(a.g_x) + row * nvec;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = v * gthreads + t;
        if (i >= nvec) break;
        float o[VEC], q[VEC];
        unpack<T, VEC>(rs_sum[v], q);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = fmaf(g[v][j] - c0 - xh[v][j] * c1, rs, q[j]);
        gx[i] = pack<T, VEC>(o);
      }
    }
  }
  if (a.part) {
    // the groups' sums, added in their order: one partial row a CTA
    __syncthreads();
    float* sums = reinterpret_cast<float*>(ring);   // [rpc][2][cols]
    float* mine = sums + (int64_t)group * 2 * a.cols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * gthreads + t;
      if (i >= nvec) break;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        mine[i * VEC + j] = gw[v][j];
        mine[a.cols + i * VEC + j] = gb[v][j];
      }
    }
    __syncthreads();
    float* pw = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    for (int c = threadIdx.x; c < 2 * (int)a.cols; c += blockDim.x) {
      float acc = sums[c];
      for (int q = 1; q < a.rpc; ++q) acc += sums[(int64_t)q * 2 * a.cols + c];
      pw[c] = acc;
    }
  }
}

// g_w (blockIdx.y = 0) and g_b (1): the partial rows of 32 columns, added in a
// fixed order.  8 loads in flight a thread (4: 0.4 us more; 10, with registers for one CTA an
// SM, 1 us more).
constexpr int kRedRows = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kRedRows)
    k_norm_bwd_reduce(const float* __restrict__ part, int64_t n_part, int64_t cols, T* g_w,
                      T* g_b) {
  __shared__ float sh[kRedRows][33];
  T* out = blockIdx.y == 0 ? g_w : g_b;
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  if (!out) return;
  float acc = 0.0f;
  if (c < cols) {
    const float* p = part + blockIdx.y * cols + c;
#pragma unroll 8
    for (int64_t r = threadIdx.y; r < n_part; r += kRedRows) acc += p[r * 2 * cols];
  }
  sh[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < kRedRows; ++i) acc += sh[i][threadIdx.x];
    out[c] = static_cast<T>(acc);
  }
}

// How a row is laid over threads: the vector width, vectors per thread, warps
// per row and rows per CTA.
struct NormShape {
  int vec, nv, wpr, rpc;
  bool full;   // 16-byte vectors
  int threads() const { return 32 * wpr * rpc; }
  int ring_ctas() const { return threads() > 256 ? 1 : threads() > 160 ? 2 : 3; }   // of an SM
};

// `narrow`: 8- and 4-byte vectors too (else single values where 16 bytes do not fit).
NormShape norm_shape(int64_t cols, int64_t x_stride, jm_dtype io, bool narrow) {
  NormShape s;
  const int full = io == JM_BF16 ? 8 : 4;
  s.vec = full;
  while (s.vec > 1 && (cols % s.vec || x_stride % s.vec)) s.vec = narrow ? s.vec / 2 : 1;
  s.full = s.vec == full;
  const int64_t nvec = cols / s.vec;
  // The fewest warps that hold the row at 2 vectors of 16 bytes a thread (more only where
  // 32 warps are not enough), or of narrower ones at 4, 8 or 16 values a thread: up to 512
  // columns as many as let one warp hold the row (16000 x 332: 11.2 us, with 3 warps and
  // their barriers 18.2 us), then 8 (816 x 943: 5.2 us, with 16 6.6 us), above 2048 16
  // (554 x 3141: 7.3 us, with 4 and 1024 threads 11.4 us).
  const int values = cols <= 128 ? 4 : cols <= 256 ? 8 : cols <= 512 ? 16 : cols <= 2048 ? 8 : 16;
  s.nv = s.full ? 2 : values / s.vec;
  int64_t wpr = (nvec + 32 * s.nv - 1) / (32 * s.nv);
  if (wpr > 32) {
    s.nv = 4;     // float32 above 8192 columns
    wpr = (nvec + 127) / 128;
  }
  s.wpr = (int)wpr;
  s.rpc = s.wpr >= 8 ? 1 : 8 / s.wpr;  // CTAs of 256 threads, or one wider row
  return s;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, cudaStream_t s, size_t smem,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename Args>
using NormKern = void (*)(const Args);

// The kernel built for a shape's threads (rounded up to 256, 512 or 1024, which sets the
// registers a thread may use): 2 vectors of 16 bytes a thread (4 only in float32 above 8192
// columns, at 1024 threads), or 4, 8 (2048 columns at most) or 16 values in narrower ones.
#define JMIX_NORM_FULL(KERN, T, FULL)                             \
  (s.threads() <= 256  ? KERN<T, FULL, 2, 256>                    \
   : s.threads() <= 512 ? KERN<T, FULL, 2, 512>                   \
                        : KERN<T, FULL, 2, 1024>)
#define JMIX_NORM_NARROW(KERN, T, VEC)                            \
  (s.nv * VEC == 4       ? KERN<T, VEC, 4 / VEC, 256>             \
   : s.nv * VEC == 8     ? KERN<T, VEC, 8 / VEC, 256>             \
   : s.threads() <= 256  ? KERN<T, VEC, 16 / VEC, 256>            \
   : s.threads() <= 512  ? KERN<T, VEC, 16 / VEC, 512>            \
                         : KERN<T, VEC, 16 / VEC, 1024>)

NormKern<NormFwdArgs> fwd_kernel(const NormShape& s, jm_dtype io) {
  if (io == JM_BF16) {
    if (s.full) return JMIX_NORM_FULL(k_norm_fwd, __nv_bfloat16, 8);
    return s.vec == 4   ? JMIX_NORM_NARROW(k_norm_fwd, __nv_bfloat16, 4)
           : s.vec == 2 ? JMIX_NORM_NARROW(k_norm_fwd, __nv_bfloat16, 2)
                        : JMIX_NORM_NARROW(k_norm_fwd, __nv_bfloat16, 1);
  }
  if (s.full) return s.nv == 4 ? k_norm_fwd<float, 4, 4, 1024> : JMIX_NORM_FULL(k_norm_fwd, float, 4);
  return s.vec == 2 ? JMIX_NORM_NARROW(k_norm_fwd, float, 2)
                    : JMIX_NORM_NARROW(k_norm_fwd, float, 1);
}

NormKern<NormBwdArgs> ring_kernel(const NormShape& s, jm_dtype io) {
  if (io == JM_BF16) {
    if (s.full) return JMIX_NORM_FULL(k_norm_bwd_ring, __nv_bfloat16, 8);
    return s.vec == 4   ? JMIX_NORM_NARROW(k_norm_bwd_ring, __nv_bfloat16, 4)
           : s.vec == 2 ? JMIX_NORM_NARROW(k_norm_bwd_ring, __nv_bfloat16, 2)
                        : JMIX_NORM_NARROW(k_norm_bwd_ring, __nv_bfloat16, 1);
  }
  if (s.full) return JMIX_NORM_FULL(k_norm_bwd_ring, float, 4);
  return s.vec == 2 ? JMIX_NORM_NARROW(k_norm_bwd_ring, float, 2)
                    : JMIX_NORM_NARROW(k_norm_bwd_ring, float, 1);
}

// (every aligned row but a float32 one above 8192 columns has a ring)
NormKern<NormBwdArgs> bwd_kernel(const NormShape& s, jm_dtype io) {
  if (io == JM_BF16) return JMIX_NORM_NARROW(k_norm_bwd, __nv_bfloat16, 1);
  return s.full ? k_norm_bwd<float, 4, 4, 1024> : JMIX_NORM_NARROW(k_norm_bwd, float, 1);
}
#undef JMIX_NORM_FULL
#undef JMIX_NORM_NARROW

size_t ring_stage(int64_t cols, bool g_sum, const NormShape& s, jm_dtype io) {
  return (size_t)ring_part_bytes((size_t)s.rpc * cols * (io == JM_BF16 ? 2 : 4), !s.full) *
         (g_sum ? 3 : 2);
}

// Stages of the backward's ring (at least 2), or 0 where the loading kernel runs: rows of
// x apart by no multiple of 16 bytes, or too long for two stages.
int ring_stages(int64_t cols, int64_t x_stride, bool g_sum, const NormShape& s, jm_dtype io) {
  if ((!s.full && x_stride != cols) || (s.full && s.nv != 2)) return 0;
  const size_t most = 220 * 1024 / s.ring_ctas();
  const int n = (int)(most / ring_stage(cols, g_sum, s, io));
  return n < 2 ? 0 : n < kNormMaxStages ? n : kNormMaxStages;
}

size_t ring_bytes(int64_t cols, bool g_sum, int stages, const NormShape& s, jm_dtype io) {
  const size_t ring = stages * ring_stage(cols, g_sum, s, io);
  const size_t sums = (size_t)s.rpc * 2 * cols * 4;
  return ring > sums ? ring : sums;
}

// CTAs of the backward: as many as are resident at once, so that there are few
// partial rows to add.
int64_t bwd_ctas(int64_t rows, const NormShape& s, bool ring) {
  const int64_t most = (int64_t)kNormSMs * (ring ? s.ring_ctas() : s.threads() > 256 ? 1 : 3);
  const int64_t need = (rows + s.rpc - 1) / s.rpc;
  return need < most ? need : most;
}

}  // namespace

size_t norm_bwd_ws_bytes(int64_t rows, int64_t cols, int64_t x_stride, jm_dtype io) {
  // partial rows of whichever kernel leaves more (which one runs depends on g_sum too)
  const NormShape r = norm_shape(cols, x_stride, io, true), s = norm_shape(cols, x_stride, io, false);
  const int64_t ring = bwd_ctas(rows, r, true), plain = bwd_ctas(rows, s, false) * s.rpc;
  return sizeof(ErrFlags) + align256((size_t)((ring > plain ? ring : plain) * 2 * cols) * 4);
}

cudaError_t run_norm_fwd(NormFwdArgs a, jm_dtype io, Problem& p) {
  const NormShape s = norm_shape(a.cols, a.x_stride, io, true);
  a.wpr = s.wpr;
  a.rpc = s.rpc;
  const int64_t ctas = (a.rows + s.rpc - 1) / s.rpc;
  launches_begin(p);
  const cudaError_t e = launch_pdl(fwd_kernel(s, io), dim3((unsigned)ctas), dim3(s.threads()),
                                   p.stream, 0, a);
  if (e == cudaSuccess) launched(p, "k_norm_fwd");
  return e;
}

cudaError_t run_norm_bwd(NormBwdArgs a, void* g_w, void* g_b, char* ws, jm_dtype io, Problem& p) {
  NormShape s = norm_shape(a.cols, a.x_stride, io, true);
  a.stages = ring_stages(a.cols, a.x_stride, a.g_sum != nullptr, s, io);
  if (a.stages == 0) s = norm_shape(a.cols, a.x_stride, io, false);
  a.wpr = s.wpr;
  a.rpc = s.rpc;
  a.err = reinterpret_cast<ErrFlags*>(ws);
  const bool sums = g_w || g_b;
  float* part = reinterpret_cast<float*>(ws + sizeof(ErrFlags));
  a.part = sums ? part : nullptr;
  const int64_t ctas = bwd_ctas(a.rows, s, a.stages > 0);
  const int64_t part_rows = a.stages > 0 ? ctas : ctas * s.rpc;
  cudaError_t e = cudaSuccess;
  launches_begin(p);
  if (ctas == 0) {
    e = cudaMemsetAsync(ws, 0, sizeof(ErrFlags), p.stream);
  } else if (a.stages > 0) {
    const NormKern<NormBwdArgs> kern = ring_kernel(s, io);
    // (a flag of the function on the current device; setting it again costs a few tenths
    // of a microsecond)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
    if (e == cudaSuccess)
      e = launch_pdl(kern, dim3((unsigned)ctas), dim3(s.threads()), p.stream,
                     ring_bytes(a.cols, a.g_sum != nullptr, a.stages, s, io), a);
    if (e == cudaSuccess) launched(p, "k_norm_bwd");
  } else {
    e = launch_pdl(bwd_kernel(s, io), dim3((unsigned)ctas), dim3(s.threads()), p.stream, 0, a);
    if (e == cudaSuccess) launched(p, "k_norm_bwd");
  }
  if (e == cudaSuccess && sums) {
    const dim3 grid((unsigned)((a.cols + 31) / 32), 2);
    if (io == JM_BF16)
      e = launch_pdl(k_norm_bwd_reduce<__nv_bfloat16>, grid, dim3(32, kRedRows), p.stream, 0,
                     (const float*)part, part_rows, a.cols, static_cast<__nv_bfloat16*>(g_w),
                     static_cast<__nv_bfloat16*>(g_b));
    else
      e = launch_pdl(k_norm_bwd_reduce<float>, grid, dim3(32, kRedRows), p.stream, 0,
                     (const float*)part, part_rows, a.cols, static_cast<float*>(g_w),
                     static_cast<float*>(g_b));
    if (e == cudaSuccess) launched(p, "k_norm_bwd_reduce");
  }
  return e;
}

}  // namespace jmix
