// A whole mixture-of-experts layer for few tokens in two kernels.
//
//   logits = x Wr^T;  the top_k experts of each token (softmax weights g)
//   h   = silu(x Wgate_e^T) (x Wup_e^T)     for each (token, chosen expert) pair
//   out = sum_i g_i h_i Wdown_{e_i}^T + residual
//
// k_moe_route: one CTA per token; logits, choice, weights.
// k_moe: one CTA per SM streams the chosen experts' weights once.  With few tokens
// those bytes bound the layer (an expert of 4096 x 14336 is 352 MB: 54 us of HBM time,
// its products for 32 tokens 7 us of tensor time), so the design keeps HBM busy:
//
// * The weights are the MMA's A operand (128 rows of weights = TMEM lanes), the tokens
//   its N: few tokens waste tensor time that is free here, and no weight is read twice.
// * A phase's work is a line of units (block of an expert's tokens, tile of weight rows)
//   x K steps of 64, cut into equal contiguous ranges, one per CTA: every SM streams the
//   same bytes whatever the number of experts in use.  A step brings 256 weight rows:
//   128 of gate and the same 128 of up in the first phase (so that h is formed in the
//   thread that holds both), 256 of down in the second.
// * A unit inside one CTA's range is finished from TMEM.  A cut one leaves float32
//   partial tiles, each CTA of it then finishing its share of the columns; partial tiles
//   are added in CTA order, so results do not depend on timing.
// * Warp 0 streams weights, warp 6 the tokens' rows (gathered by index, then rows of h),
//   warp 1 issues the MMAs, warps 2-5 drain them.  Nothing but warp 6 waits between the
//   phases, and only for h of the block it needs, so the ring is full of
//   down-projection weights when h arrives.
//
// CTAs wait for one another (partial tiles, h, the last sum), so the launch is
// cooperative; every wait is bounded and reports to the error header.
#include <cuda.h>

#include "block_epilogue.cuh"
#include "jmix_internal.cuh"
#include "sm100.cuh"

namespace jmix {
namespace {

using namespace sm100;

constexpr int kThreads = 224;
constexpr int kWarps = kThreads / 32;
constexpr int kRouteThreads = 512;
constexpr int kK = 64;                          // K per step: one 128-byte swizzle span
constexpr int kSlabBytes = 128 * kK * 2;        // 128 weight rows
constexpr int kWBytes = 2 * kSlabBytes;         // weights of a step
constexpr int kMaxCtas = 148;
constexpr int kMaxTokens = 256, kMaxTopK = 8, kMaxExperts = 256;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kMaxBlock = 128;                  // token rows per unit
constexpr int kMaxEntries = kMaxExperts + kMaxPairs / 16;
constexpr int kMaxStages = 8;

// A block of the token rows of an expert: pair rows [r0, r0 + n).
struct Entry {
  uint16_t e, r0, n, pad;
};

// Routing lists, rebuilt by every CTA in shared memory.  Pair rows (token, choice) are
// sorted by expert, tokens ascending.
struct Lists {
  Entry entry[kMaxEntries];
  uint16_t token[kMaxPairs];     // of a pair row
  uint16_t ent[kMaxPairs];       // block of a pair row
  uint16_t row[kMaxPairs];       // pair row of token * top_k + choice
  int count[kMaxExperts];
  int first[kMaxExperts];        // first pair row of an expert
  int n_entries;
};

// Counters that k_moe_route clears.
struct Sync {
  unsigned unit[kMaxCtas];       // steps of the cut unit that starts in a CTA's range, stored
  unsigned ready[kMaxEntries];   // steps of a block whose h is stored
  unsigned done;                 // CTAs whose second phase is stored
};

struct MoeKArgs {
  int T, E, topk, D, F, NB, stages, topk_softmax;
  const __nv_bfloat16* x;
  const __nv_bfloat16* wr;
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  int* user_idx;
  float* user_w;
  int* idx;             // [T * topk]
  float* wgt;           // [T * topk]
  __nv_bfloat16* h;     // [T * topk][F]
  float* y;             // [T * topk][tiles * 256] second products of uncut units
  float* part;          // [phase][CTA][head, tail][NB][256] partial tiles of cut units
  Sync* sync;
  ErrFlags* err;
};

// A phase's line of work, cut between `ctas` CTAs.
struct Line {
  unsigned tiles, ksteps, total, ctas;
  __device__ __forceinline__ unsigned start(unsigned c) const {
    return (unsigned)((uint64_t)total * min(c, ctas) / ctas);
  }
  // the CTA whose range holds step s (total * ctas < 2^32, checked on the host)
  __device__ __forceinline__ unsigned cta_of(unsigned s) const {
    return ((s + 1) * ctas - 1) / total;
  }
};

// No more CTAs than steps, so that no range between two others is empty.
__device__ __forceinline__ Line make_line(unsigned entries, unsigned rows, unsigned kdim,
                                          unsigned tile_rows) {
  Line l;
  l.tiles = (rows + tile_rows - 1) / tile_rows;
  l.ksteps = (kdim + kK - 1) / kK;
  l.total = entries * l.tiles * l.ksteps;
  l.ctas = max(min(gridDim.x, l.total), 1u);
  return l;
}

// ------------------------------------------------------ counters between CTAs
__device__ __forceinline__ void add_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__device__ __forceinline__ bool wait_count(unsigned* p, unsigned n, ErrFlags* err, unsigned site) {
  const uint64_t t0 = globaltimer_ns();
  for (unsigned i = 0;; ++i) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    if (v >= n) return true;
    if ((i & 63) == 63 && globaltimer_ns() - t0 > kWaitLimitNs) {
      if (atomicExch(&err->timeout, 1u) == 0u) err->where = site;
      return false;
    }
  }
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Drain warps: counts `v` after all of their earlier writes.
__device__ __forceinline__ void epi_add(unsigned* p, unsigned v, int et) {
  __threadfence();
  epi_sync();
  if (et == 0) add_release(p, v);
}

__device__ __forceinline__ bool epi_wait(unsigned* p, unsigned n, ErrFlags* err, unsigned site,
                                         int et, int* flag) {
  if (et == 0) *flag = wait_count(p, n, err, site) ? 1 : 0;
  epi_sync();
  const bool ok = *flag != 0;
  epi_sync();
  return ok;
}

// ------------------------------------------------------------------- routing

// a is a better choice than b: larger (NaN is largest), lower index on a tie.
__device__ __forceinline__ bool better(double a, int ia, double b, int ib) {
  const bool na = a != a, nb = b != b;
  if (na != nb) return na;
  if (!na && a != b) return a > b;
  return ia < ib;
}

// One warp: the top_k of a token's logits and their softmax weights.
__device__ void token_choice(const MoeKArgs& a, int t, const double* logits) {
  const int lane = threadIdx.x & 31;
  unsigned taken = 0;   // this lane's experts lane, lane + 32, ... already chosen
  double top = 0.0;
  float mine = 0.0f, sum = 0.0f;
  for (int i = 0; i < a.topk; ++i) {
    double v = 0.0;
    int at = 1 << 30;
    for (int j = 0, e = lane; e < a.E; ++j, e += 32)
      if (!(taken >> j & 1u) && (at == 1 << 30 || better(logits[e], e, v, at))) {
        v = logits[e];
        at = e;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, v, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (oa != 1 << 30 && (at == 1 << 30 || better(ov, oa, v, at))) {
        v = ov;
        at = oa;
      }
    }
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    if (i == 0) top = v;
    const float ex = expf((float)(v - top));
    sum += ex;
    if (lane == i) {
      mine = ex;
      a.idx[t * a.topk + i] = at;
      if (a.user_idx) a.user_idx[t * a.topk + i] = at;
    }
  }
  if (!a.topk_softmax) {
    sum = 0.0f;
    for (int e = lane; e < a.E; e += 32) sum += expf((float)(logits[e] - top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if (lane < a.topk) {
    a.wgt[t * a.topk + lane] = mine / sum;
    if (a.user_w) a.user_w[t * a.topk + lane] = mine / sum;
  }
}

// Logits: products of bf16 are exact in float32; 8 of them are added in float32 and the
// sums in float64, so that close logits keep their order.
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(const MoeKArgs a) {
  __shared__ double logits[kMaxExperts];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  if (t == 0) {
    unsigned* s = reinterpret_cast<unsigned*>(a.sync);
    for (unsigned i = threadIdx.x; i < sizeof(Sync) / 4; i += kRouteThreads) s[i] = 0u;
    if (threadIdx.x < sizeof(ErrFlags) / 4) reinterpret_cast<unsigned*>(a.err)[threadIdx.x] = 0u;
  }
  const int n8 = a.D / 8;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x) + (int64_t)t * n8;
  for (int e = warp; e < a.E; e += kRouteThreads / 32) {
    const uint4* wr = reinterpret_cast<const uint4*>(a.wr) + (int64_t)e * n8;
    double acc = 0.0;
#pragma unroll 8
    for (int i = lane; i < n8; i += 32) {
      float xv[8], wv[8], s = 0.0f;
      unpack8(xr[i], xv);
      unpack8(__ldg(wr + i), wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(xv[j], wv[j], s);
      acc += (double)s;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) logits[e] = acc;
  }
  __syncthreads();
  if (warp == 0) token_choice(a, t, logits);
}

// The lists of every CTA from the choices.
__device__ void build_lists(const MoeKArgs& a, Lists& L) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = a.T * a.topk;
  for (int e = tid; e < a.E; e += kThreads) L.count[e] = 0;
  __syncthreads();
  for (int p = tid; p < P; p += kThreads) {
    const int e = a.idx[p];
    L.ent[p] = (uint16_t)e;          // expert of the pair, until the blocks are known
    atomicAdd(&L.count[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kThreads) {
    int first = 0, at = 0;
    for (int q = 0; q < e; ++q) {
      first += L.count[q];
      at += (L.count[q] + a.NB - 1) / a.NB;
    }
    const int n = L.count[e];
    L.first[e] = first;
    for (int r = 0; r < n; r += a.NB, ++at)
      L.entry[at] = {(uint16_t)e, (uint16_t)(first + r), (uint16_t)min(a.NB, n - r), 0};
    if (e == a.E - 1) L.n_entries = at;
  }
  __syncthreads();
  // pairs of an expert in order of their token: a warp per expert in use
  for (int e = warp; e < a.E; e += kWarps) {
    if (L.count[e] == 0) continue;
    int at = L.first[e];
    for (int p0 = 0; p0 < P; p0 += 32) {
      const int p = p0 + lane;
      const bool hit = p < P && L.ent[p] == e;
      const unsigned m = __ballot_sync(0xffffffffu, hit);
      if (hit) {
        const int r = at + __popc(m & ((1u << lane) - 1u));
        L.token[r] = (uint16_t)(p / a.topk);
        L.row[p] = (uint16_t)r;
      }
      at += __popc(m);
    }
  }
  __syncthreads();
  for (int i = warp; i < L.n_entries; i += kWarps)
    for (int r = lane; r < L.entry[i].n; r += 32) L.ent[L.entry[i].r0 + r] = (uint16_t)i;
  __syncthreads();
}

// Partial tile of CTA `cta` in phase `ph`: of the unit that starts before its range
// (slot 0) or in it (slot 1).  Rows of 256 floats, one per token row of the block.
__device__ __forceinline__ float* part_of(const MoeKArgs& a, int ph, unsigned cta, int slot) {
  return a.part + ((int64_t)((ph * kMaxCtas + cta) * 2 + slot) * a.NB) * 256;
}

__device__ __forceinline__ float4 ld4(const float* p) {
  return __ldcg(reinterpret_cast<const float4*>(p));
}

__device__ __forceinline__ void add4(float4& v, const float4& q) {
  v.x += q.x;
  v.y += q.y;
  v.z += q.z;
  v.w += q.w;
}

// silu(g) u
__device__ __forceinline__ float glu(float g, float u) { return act_apply(g, JM_ACT_SILU) * u; }

// This CTA's share of a cut unit's h: partial tiles of CTAs c0..c1 in that order.
__device__ void join_h(const MoeKArgs& a, const Entry& en, unsigned tile, unsigned c0, unsigned c1,
                       int et) {
  const unsigned nseg = c1 - c0 + 1, total = en.n * 32u;
  for (unsigned i = (blockIdx.x - c0) * 128 + et; i < total; i += nseg * 128) {
    const unsigned r = i >> 5, f = (i & 31) * 4, col = tile * 128 + f;
    if (col >= (unsigned)a.F) continue;
    const float* p = part_of(a, 0, c0, 1) + r * 256 + f;
    float4 g = ld4(p), u = ld4(p + 128);
    for (unsigned c = c0 + 1; c <= c1; ++c) {
      p = part_of(a, 0, c, 0) + r * 256 + f;
      add4(g, ld4(p));
      add4(u, ld4(p + 128));
    }
    *reinterpret_cast<uint2*>(a.h + (int64_t)(en.r0 + r) * a.F + col) =
        make_uint2(pack2(glu(g.x, u.x), glu(g.y, u.y)), pack2(glu(g.z, u.z), glu(g.w, u.w)));
  }
}

// out of every token: its experts' products weighted in the order of the choices.
__device__ void form_out(const MoeKArgs& a, const Lists& L, const Line& l, int et) {
  const unsigned d4 = (unsigned)a.D / 4, total = (unsigned)a.T * d4;
  const int64_t width = (int64_t)l.tiles * 256;
  for (unsigned i = blockIdx.x * 128 + et; i < total; i += gridDim.x * 128) {
    const unsigned t = i / d4, d = (i - t * d4) * 4, tile = d >> 8, in = d & 255;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = 0; c < a.topk; ++c) {
      const unsigned p = t * a.topk + c;
      const int r = L.row[p], ent = L.ent[r];
      const float w = a.wgt[p];
      const unsigned s0 = (ent * l.tiles + tile) * l.ksteps;
      const unsigned c0 = l.cta_of(s0), c1 = l.cta_of(s0 + l.ksteps - 1);
      float4 v;
      if (c0 == c1) {
        v = ld4(a.y + r * width + d);
      } else {
        const int64_t at = (int64_t)(r - L.entry[ent].r0) * 256 + in;
        v = ld4(part_of(a, 1, c0, 1) + at);
        for (unsigned q = c0 + 1; q <= c1; ++q) add4(v, ld4(part_of(a, 1, q, 0) + at));
      }
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    const int64_t at = (int64_t)t * a.D + d;
    if (a.residual) {
      const uint2 q = *reinterpret_cast<const uint2*>(a.residual + at);
      o.x += __uint_as_float(q.x << 16);
      o.y += __uint_as_float(q.x & 0xffff0000u);
      o.z += __uint_as_float(q.y << 16);
      o.w += __uint_as_float(q.y & 0xffff0000u);
    }
    *reinterpret_cast<uint2*>(a.out + at) = make_uint2(pack2(o.x, o.y), pack2(o.z, o.w));
  }
}

// tm_wg, tm_wu gate and up [E][F][D], tm_wd down [E][D][F], tm_x tokens by row index,
// tm_h rows of h.
__global__ void __launch_bounds__(kThreads, 1)
    k_moe(const __grid_constant__ CUtensorMap tm_wg, const __grid_constant__ CUtensorMap tm_wu,
          const __grid_constant__ CUtensorMap tm_wd, const __grid_constant__ CUtensorMap tm_x,
          const __grid_constant__ CUtensorMap tm_h, const MoeKArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int S = a.stages;
  const int stage_bytes = kWBytes + a.NB * 128;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int epi_flag;
  Lists& L = *reinterpret_cast<Lists*>(smem + S * stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t tmem_cols = 4 * a.NB;   // two accumulators of two row groups: 64..512

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 2);    // weights' and tokens' producers
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 4);
    }
    fence_mbar_init();
    prefetch_tmap(&tm_wg);
    prefetch_tmap(&tm_wu);
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_wd);
    prefetch_tmap(&tm_h);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  grid_dep_wait();
  build_lists(a, L);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const Line line[2] = {make_line(L.n_entries, a.F, a.D, 128), make_line(L.n_entries, a.D, a.F, 256)};

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = l2_evict_first_policy();   // weights pass through once
      unsigned it = 0;
      bool ok = true;
      for (int ph = 0; ok && ph < 2; ++ph) {
        const Line& l = line[ph];
        const unsigned s1 = l.start(blockIdx.x + 1);
        for (unsigned s = l.start(blockIdx.x); s < s1; ++s, ++it) {
          const unsigned u = s / l.ksteps, ent = u / l.tiles;
          const int k = (int)(s - u * l.ksteps) * kK, tile = (int)(u - ent * l.tiles);
          const int e = L.entry[ent].e;
          const unsigned st = it % S;
          if (it >= (unsigned)S &&
              !mbar_wait(smem_u32(&empty[st]), ((it / S) - 1) & 1u, a.err, 92)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full[st]), dst = smem_u32(smem + st * stage_bytes);
          mbar_arrive_expect_tx(fb, kWBytes);
          if (ph == 0) {
            tma_load_3d(dst, &tm_wg, fb, k, tile * 128, e, pol);
            tma_load_3d(dst + kSlabBytes, &tm_wu, fb, k, tile * 128, e, pol);
          } else {
            tma_load_3d(dst, &tm_wd, fb, k, tile * 256, e, pol);
            tma_load_3d(dst + kSlabBytes, &tm_wd, fb, k, tile * 256 + 128, e, pol);
          }
        }
      }
    }
  } else if (warp == 6) {
    unsigned it = 0;
    bool ok = true;
    for (int ph = 0; ok && ph < 2; ++ph) {
      const Line& l = line[ph];
      const unsigned s1 = l.start(blockIdx.x + 1);
      unsigned ready = ~0u;   // the block whose h is known to be there
      for (unsigned s = l.start(blockIdx.x); s < s1; ++s, ++it) {
        const unsigned u = s / l.ksteps, ent = u / l.tiles;
        const int k = (int)(s - u * l.ksteps) * kK;
        const Entry en = L.entry[ent];
        const int n16 = (en.n + 15) / 16;
        const unsigned st = it % S;
        int w = 1;
        if (lane == 0) {
          if (ph == 1 && ent != ready)
            w = wait_count(&a.sync->ready[ent], line[0].tiles * line[0].ksteps, a.err, 93) ? 1 : 0;
          if (w && it >= (unsigned)S)
            w = mbar_wait(smem_u32(&empty[st]), ((it / S) - 1) & 1u, a.err, 94) ? 1 : 0;
        }
        if (__shfl_sync(0xffffffffu, w, 0) == 0) {
          ok = false;
          break;
        }
        __syncwarp();
        if (ph == 1 && ent != ready) {
          fence_proxy_async_global();
          ready = ent;
        }
        const uint32_t fb = smem_u32(&full[st]);
        const uint32_t dst = smem_u32(smem + st * stage_bytes + kWBytes);
        if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)(n16 * 16 * 128));
        __syncwarp();
        if (ph == 0) {
          // 4 rows by index at a time; rows behind the last repeat it (their columns of
          // the accumulator are not read)
          for (int r = lane * 4; r < n16 * 16; r += 128) {
            int t[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = L.token[en.r0 + min(r + j, en.n - 1)];
            tma_gather4(dst + r * 128, &tm_x, fb, k, t[0], t[1], t[2], t[3]);
          }
        } else if (lane < n16) {
          tma_load_2d(dst + lane * 2048, &tm_h, fb, k, en.r0 + lane * 16);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      unsigned it = 0, j = 0;
      bool ok = true;
      for (int ph = 0; ok && ph < 2; ++ph) {
        const Line& l = line[ph];
        const unsigned s1 = l.start(blockIdx.x + 1);
        for (unsigned s = l.start(blockIdx.x); ok && s < s1; ++j) {
          const unsigned u = s / l.ksteps, end = min(s1, (u + 1) * l.ksteps);
          const int n16 = (L.entry[u / l.tiles].n + 15) / 16;
          const uint32_t idesc = idesc_bf16_f32(128, n16 * 16);
          const unsigned b = j & 1;
          if (j >= 2 && !mbar_wait(smem_u32(&acc_empty[b]), ((j >> 1) - 1) & 1u, a.err, 95)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + b * (uint32_t)(2 * a.NB);
          for (const unsigned first = s; s < end; ++s, ++it) {
            const unsigned st = it % S;
            if (!mbar_wait(smem_u32(&full[st]), (it / S) & 1u, a.err, 96)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t wa = smem_u32(smem + st * stage_bytes), xb = wa + kWBytes;
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int kk = 0; kk < kK / 16; ++kk)
                umma_f16(d + (uint32_t)(g * a.NB),
                         sw128_kmajor_desc(wa + g * kSlabBytes + kk * 32),
                         sw128_kmajor_desc(xb + kk * 32), idesc, (s > first || kk > 0) ? 1u : 0u);
            umma_commit(smem_u32(&empty[st]));
          }
          if (ok) umma_commit(smem_u32(&acc_full[b]));
        }
      }
    }
  } else {
    const int lg = warp & 3, et = lg * 32 + lane;   // TMEM lane = weight row of a group
    unsigned j = 0;
    bool ok = true;
    for (int ph = 0; ok && ph < 2; ++ph) {
      const Line& l = line[ph];
      const unsigned s0 = l.start(blockIdx.x), s1 = l.start(blockIdx.x + 1);
      for (unsigned s = s0; s < s1; ++j) {
        const unsigned u = s / l.ksteps, u0 = u * l.ksteps, end = min(s1, u0 + l.ksteps);
        const unsigned ent = u / l.tiles, tile = u - ent * l.tiles;
        const bool whole = s == u0 && end == u0 + l.ksteps;
        const Entry en = L.entry[ent];
        const unsigned b = j & 1;
        if (!mbar_wait(smem_u32(&acc_full[b]), (j >> 1) & 1u, a.err, 97)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem + ((uint32_t)(lg * 32) << 16) + b * (uint32_t)(2 * a.NB);
        float* dst = part_of(a, ph, blockIdx.x, s == u0 ? 1 : 0) + et;
        int64_t pitch = 256;
        if (ph == 1 && whole) {
          pitch = (int64_t)l.tiles * 256;
          dst = a.y + en.r0 * pitch + tile * 256 + et;
        }
        const unsigned f = tile * 128 + et;
        for (int c = 0; c < en.n; c += 16) {
          uint32_t g[16], q[16];
          tmem_ld16(tb + c, g);
          tmem_ld16(tb + a.NB + c, q);
          tmem_ld_wait();
          if (ph == 0 && whole) {
            if (f < (unsigned)a.F) {
              __nv_bfloat16* hp = a.h + (int64_t)(en.r0 + c) * a.F + f;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (c + i < en.n)
                  hp[(int64_t)i * a.F] =
                      __float2bfloat16_rn(glu(__uint_as_float(g[i]), __uint_as_float(q[i])));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + i < en.n) {
                __stcg(dst + (c + i) * pitch, __uint_as_float(g[i]));
                __stcg(dst + (c + i) * pitch + 128, __uint_as_float(q[i]));
              }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&acc_empty[b]));
        if (ph == 0) {
          if (whole) {
            fence_proxy_async_global();   // h is read by TMA
            epi_add(&a.sync->ready[ent], l.ksteps, et);
          } else {
            epi_add(&a.sync->unit[l.cta_of(u0)], end - s, et);
          }
        }
        s = end;
      }
      if (ph == 0) {
        // this CTA's share of the cut units it took part in (its first and its last),
        // after all that others wait for is stored
        for (unsigned s = s0; ok && s < s1;) {
          const unsigned u = s / l.ksteps, u0 = u * l.ksteps, end = min(s1, u0 + l.ksteps);
          const unsigned ent = u / l.tiles;
          if (s != u0 || end != u0 + l.ksteps) {
            const unsigned c0 = l.cta_of(u0), c1 = l.cta_of(u0 + l.ksteps - 1);
            ok = epi_wait(&a.sync->unit[c0], l.ksteps, a.err, 98, et, &epi_flag);
            if (ok) {
              join_h(a, L.entry[ent], u - ent * l.tiles, c0, c1, et);
              fence_proxy_async_global();
              epi_add(&a.sync->ready[ent], end - s, et);
            }
          }
          s = end;
        }
      }
    }
    epi_add(&a.sync->done, 1, et);
    if (epi_wait(&a.sync->done, gridDim.x, a.err, 99, et, &epi_flag))
      form_out(a, L, line[1], et);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// ------------------------------------------------------------------ host side

// A row-major bf16 tensor [n][rows][inner] as swizzled boxes of 64 inner values.
bool map3(CUtensorMap* m, const void* base, int64_t n, int64_t rows, int64_t inner) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)n};
  cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)(inner * rows) * 2};
  cuuint32_t bx[3] = {kK, 128, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map2(CUtensorMap* m, const void* base, int64_t rows, int64_t inner, int box) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)inner * 2};
  cuuint32_t bx[2] = {kK, (cuuint32_t)box}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Token rows a unit holds.  An expert with more rows streams its weights again for the
// next block, so the block has room for twice the mean (and 16) of an even router; more
// room would only take shared memory from the weights' ring.
int moe_block(int64_t T, int64_t E, int64_t k) {
  int64_t want = 2 * ceil_div(T * k, E) + 16;
  if (want > T) want = T;
  int nb = 16;
  while (nb < want && nb < kMaxBlock) nb *= 2;
  return nb;
}

constexpr size_t kSmemMost = 227 * 1024;
constexpr size_t kStaticMost = 512;   // barriers and flags
constexpr size_t kListBytes = (sizeof(Lists) + 255) / 256 * 256;

int ring_stages(int nb) {
  const size_t n = (kSmemMost - kStaticMost - 1024 - kListBytes) / (kWBytes + nb * 128);
  return n > kMaxStages ? kMaxStages : (int)n;
}

size_t ring_smem(int nb) {
  return 1024 + ring_stages(nb) * (size_t)(kWBytes + nb * 128) + kListBytes;
}

struct MoeWs {
  Sync* sync;
  int* idx;
  float* wgt;
  __nv_bfloat16* h;
  float* y;
  float* part;
  size_t bytes;
};

MoeWs moe_ws(const MoeArgs& m, char* base) {
  MoeWs w{};
  size_t off = sizeof(ErrFlags);
  auto take = [&](size_t n) {
    char* p = base ? base + off : nullptr;
    off += align256(n);
    return p;
  };
  const int64_t P = m.T * m.topk, nb = moe_block(m.T, m.E, m.topk);
  w.sync = reinterpret_cast<Sync*>(take(sizeof(Sync)));
  w.idx = reinterpret_cast<int*>(take((size_t)P * 4));
  w.wgt = reinterpret_cast<float*>(take((size_t)P * 4));
  w.h = reinterpret_cast<__nv_bfloat16*>(take((size_t)P * m.F * 2));
  w.y = reinterpret_cast<float*>(take((size_t)P * ceil_div(m.D, 256) * 256 * 4));
  w.part = reinterpret_cast<float*>(take(P ? (size_t)4 * kMaxCtas * nb * 256 * 4 : 0));
  w.bytes = off;
  return w;
}

// The steps of the longer line, at most.
int64_t most_steps(const MoeArgs& m) {
  const int64_t P = m.T * m.topk, nb = moe_block(m.T, m.E, m.topk);
  const int64_t entries = (m.E < P ? m.E : P) + P / nb;
  const int64_t a = ceil_div(m.F, 128) * ceil_div(m.D, kK);
  const int64_t b = ceil_div(m.D, 256) * ceil_div(m.F, kK);
  return entries * (a > b ? a : b);
}

// CTAs of k_moe: one per SM.
int moe_ctas() {
  static std::atomic<int> cache[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (cudaFuncSetAttribute(k_moe, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)(kSmemMost - kStaticMost)) != cudaSuccess)
    return 0;
  if (n > kMaxCtas) n = kMaxCtas;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace

bool moe_fits(const MoeArgs& m) { return (double)most_steps(m) * kMaxCtas < 4.0e9; }

size_t moe_ws_bytes(const MoeArgs& m) { return moe_ws(m, nullptr).bytes; }

cudaError_t run_moe(const MoeArgs& m, Problem& p) {
  const MoeWs w = moe_ws(m, m.ws);
  const int ctas = moe_ctas();
  if (ctas <= 0) return cudaErrorInvalidConfiguration;
  MoeKArgs a{};
  a.T = (int)m.T;
  a.E = (int)m.E;
  a.topk = (int)m.topk;
  a.D = (int)m.D;
  a.F = (int)m.F;
  a.NB = moe_block(m.T, m.E, m.topk);
  a.stages = ring_stages(a.NB);
  a.topk_softmax = m.topk_softmax;
  a.x = static_cast<const __nv_bfloat16*>(m.x);
  a.wr = static_cast<const __nv_bfloat16*>(m.router_w);
  a.residual = static_cast<const __nv_bfloat16*>(m.residual);
  a.out = static_cast<__nv_bfloat16*>(m.out);
  a.user_idx = m.topk_idx;
  a.user_w = m.topk_w;
  a.idx = w.idx;
  a.wgt = w.wgt;
  a.h = w.h;
  a.y = w.y;
  a.part = w.part;
  a.sync = w.sync;
  a.err = reinterpret_cast<ErrFlags*>(m.ws);
  CUtensorMap wg, wu, wd, tx, th;
  if (!map3(&wg, m.w_gate, m.E, m.F, m.D) || !map3(&wu, m.w_up, m.E, m.F, m.D) ||
      !map3(&wd, m.w_down, m.E, m.D, m.F) || !map2(&tx, m.x, m.T, m.D, 1) ||
      !map2(&th, w.h, m.T * m.topk, m.F, 16))
    return cudaErrorInvalidValue;
  launches_begin(p);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.stream = p.stream;
  cfg.gridDim = dim3((unsigned)m.T);
  cfg.blockDim = dim3(kRouteThreads);
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_moe_route, a);
  if (e != cudaSuccess) return e;
  launched(p, "k_moe_route");
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = ring_smem(a.NB);
  cfg.attrs = attr + 1;
  e = cudaLaunchKernelEx(&cfg, k_moe, wg, wu, wd, tx, th, a);
  if (e == cudaSuccess) launched(p, "k_moe");
  return e;
}

}  // namespace jmix
