// The epilogue of the block's matrix products (bias, activation, residual, stores of 8
// columns) and the host-side tensor-map encoder they share.
#pragma once

#include <cuda.h>

#include <atomic>

#include "block_math.cuh"
#include "jmix_internal.cuh"

namespace jmix {

struct Epilogue {
  const __nv_bfloat16* bias;      // [N] or null
  const __nv_bfloat16* residual;  // [M, N] or null
  __nv_bfloat16* out;             // [M, N]
  __nv_bfloat16* pre;             // [M, N] or null
  int act;
};

// The few-row products of k_linear_few.cu: C[T, N] = x [T, K] . w^T with the epilogue, w
// stored [N, K], or [K, N] with w_mn.  apart: the kernel before it on the stream writes nothing
// that this one touches, and its end may be waited for at this one's end.
bool linear_few(int64_t rows, int64_t contracted);
cudaError_t run_linear_few(int64_t T, int64_t N, int64_t K, const void* x, const void* w, bool w_mn,
                           const Epilogue& ep, ErrFlags* err, bool clear_err, bool apart, Problem& p);

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Bias, activation and residual on 8 consecutive columns of one row, and the stores.
__device__ __forceinline__ void finish8(const Epilogue& e, float (&v)[8], int64_t at, int64_t col) {
  if (e.bias) {
    float b[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(e.bias + col)), b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
  }
  if (e.pre) *reinterpret_cast<uint4*>(e.pre + at) = pack8(v);
  if (e.act != JM_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_apply(v[j], e.act);
  }
  if (e.residual) {
    float r[8];
    unpack8(*reinterpret_cast<const uint4*>(e.residual + at), r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  }
  *reinterpret_cast<uint4*>(e.out + at) = pack8(v);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn tensor_map_encoder() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load(std::memory_order_relaxed);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      f = reinterpret_cast<EncodeTiledFn>(p);
    fn.store(f, std::memory_order_relaxed);
  }
  return f;
}

}  // namespace jmix
