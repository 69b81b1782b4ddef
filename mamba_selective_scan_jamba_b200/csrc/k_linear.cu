// Linear layers of the decoder block on tcgen05 tensor cores:
//   forward   out = act(x w^T + bias) + residual
//   backward  g_p = g_out act'(p);  g_x = g_p w;  g_w = g_p^T x;  g_bias = sum g_p
//
// All three products are C[M, N] = sum_k A[m, k] B[n, k] with bf16 operands and
// float32 accumulation in TMEM; they differ in which index of an operand is
// contiguous in memory:
//   forward  A = x   [m, k] K-major,            B = w   [n, k] K-major
//   g_x      A = g_p [m, n] K-major,            B = w   [n, k] read as B[k, n]: MN-major
//   g_w      A = g_p [m, n] read as A[n, m]: MN-major,  B = x [m, k] read as B[k, m]: MN-major
// tcgen05 takes either major order from a 128-byte-swizzled tile, so nothing is
// transposed in memory.
//
// k_linear_pair: persistent CTA pairs (cta_group::2), a 256 x BN tile per pair, 64-wide K
// chunks in a TMA ring, the leader issues the MMAs, each CTA drains its 128 rows from one
// of two accumulators while the next tile fills the other.  Eight warps drain: a tile of
// 256 x 256 takes the tensor cores 17 us at K 4096 but 7 us at K 1744, and one warp for
// each quarter of the TMEM lanes needed 20 us with an activation (6063 x 1744 x 8952 with
// SiLU: 322 us, with eight and staged stores 145 us).  They stage 64 columns at a time in
// swizzled shared memory, two buffers a group; the residual comes into the same place by
// TMA before the accumulator is complete, and TMA stores write whole lines.
//
// Problems with few tiles are cut along K.  Two pairs of a cluster may share a tile
// (`cpairs`): each writes the other's half of the columns, float32, into the other's shared
// memory and finishes its own (256 x 8192 x 4096 with the residual: 20.1 us; with whole
// tiles left for the other to read 21.3 us, 2 us of them these reads).  Where more cuts pay
// (`splits`), partial tiles go through global memory and k_linear_reduce adds them.
// Products of few rows are k_linear_few's.
#include <cuda.h>

#include <atomic>

#include "block_epilogue.cuh"
#include "block_math.cuh"
#include "jmix_internal.cuh"
#include "sm100.cuh"

namespace jmix {
namespace {

using namespace sm100;

constexpr int kK = 64;              // K chunk: one 128-byte swizzle atom of bf16
constexpr int kHalf = 128;          // tile rows per CTA
constexpr int kThreads = 320;      // producer, MMA and 8 epilogue warps
constexpr int kOutBytes = kHalf * 128;  // a staging buffer: 128 rows x 128 bytes
constexpr int kGroupM = 16;         // row tiles per raster group
constexpr uint32_t kTmemCols = 512;
constexpr int kABytes = kHalf * kK * 2;                      // 16 KB
constexpr int b_bytes(int BN) { return BN / 2 * kK * 2; }    // 16 or 8 KB
constexpr int stage_bytes(int BN) { return kABytes + b_bytes(BN); }
// Ring stages and staging share 224 KB.  A CTA with one tile has nothing to drain while its
// ring is in use: its ring takes all of it and the staging the ring's place afterwards
// (loads from HBM take 1.4 us under load, five stages of a 0.27 us step).
constexpr int kRegion = 224 * 1024;
constexpr int kMaxStages = kRegion / stage_bytes(128);
constexpr int kStaging = 4 * kOutBytes;
// (the half tile that the other pair of a cluster sends lies behind the ring)
constexpr int joined_bytes(int BN) { return BN / 2 * kHalf * 4; }
constexpr int stages(int BN, bool single, bool joined) {
  return (single ? kRegion - (joined ? joined_bytes(BN) : 0) : kRegion - kStaging) / stage_bytes(BN);
}
constexpr int kSmemBytes = 1024 + kRegion + 8 * (2 * kMaxStages + 6) + 16;

struct PairArgs {
  int64_t M, N, K;
  unsigned m_tiles, n_tiles;
  int cpairs;    // pairs of a cluster (1 or 2), each a range of the tile's K
  int splits;    // above 1 (cpairs 1): float32 partial tiles [splits][M][N] through tm_out
  Epilogue ep;   // (its out and residual are reached through the maps)
  ErrFlags* err;
  bool single;     // no CTA has two tiles
  bool clear_err;  // the first kernel of a call clears the error header
  // The kernel before this one writes nothing that this one reads or writes, and has itself
  // waited for all that came before: its end is waited for at this kernel's end, so that the
  // two overlap.
  bool late_wait;
};

__device__ __forceinline__ void group_sync(int grp) {
  asm volatile("bar.sync %0, 128;" ::"r"(grp + 1) : "memory");
}

__device__ __forceinline__ uint4 pack8_bits(const uint32_t* v) {
  return make_uint4(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                    pack2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                    pack2(__uint_as_float(v[4]), __uint_as_float(v[5])),
                    pack2(__uint_as_float(v[6]), __uint_as_float(v[7])));
}

template <int ACT>
__device__ __forceinline__ void apply_one(uint32_t (&v)[64]) {
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __float_as_uint(act_apply(__uint_as_float(v[i]), ACT));
}

__device__ __forceinline__ void apply_act(uint32_t (&v)[64], int act) {
  if (act == JM_ACT_RELU) apply_one<JM_ACT_RELU>(v);
  if (act == JM_ACT_GELU) apply_one<JM_ACT_GELU>(v);
  if (act == JM_ACT_SILU) apply_one<JM_ACT_SILU>(v);
}

struct Item {
  unsigned mt, nt, split;
  int k0, k1;    // K chunks [k0, k1)
};

// (32-bit throughout: a 64-bit division is several hundred cycles of one thread)
__device__ __forceinline__ Item item_of(const PairArgs& g, unsigned w, int kchunks) {
  Item it;
  const unsigned tiles = g.m_tiles * g.n_tiles;
  it.split = g.splits > 1 ? w / tiles : 0u;
  const unsigned t = w - it.split * tiles;
  const unsigned per_group = (unsigned)kGroupM * g.n_tiles;
  const unsigned grp = t / per_group, idx = t - grp * per_group;
  const unsigned rows = min((unsigned)kGroupM, g.m_tiles - grp * kGroupM);
  it.nt = idx / rows;
  it.mt = grp * kGroupM + idx - it.nt * rows;
  it.k0 = 0;
  it.k1 = kchunks;
  const int cuts = g.splits > 1 ? g.splits : g.cpairs;
  if (cuts > 1) {
    const int cut = g.splits > 1 ? (int)it.split : (int)(cluster_rank() >> 1);
    it.k0 = (int)((int64_t)kchunks * cut / cuts);
    it.k1 = (int)((int64_t)kchunks * (cut + 1) / cuts);
  }
  return it;
}

// A place in the ring and the parity of its round: counted on, since a division by the
// number of stages in each step of one thread's loop is time that the loads do not have.
struct Place {
  int n, s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ explicit Place(int n) : n(n) {}
  __device__ __forceinline__ void next() {
    if (++s == n) {
      s = 0;
      parity ^= 1u;
    }
  }
};

// What an epilogue group does with 64 columns (32 of a partial tile) of its rows.
struct Drain {
  const PairArgs& g;
  uint8_t* stage;      // two buffers, used in turn
  const int sw, grp;   // the swizzle of this thread's row
  const uint32_t res_bar;
  const int row_at;
  const bool first;    // the thread that issues the group's copies
  uint32_t res_parity = 0;
  int buf = 0;
  bool ok = true;
  __nv_bfloat16* bias;   // shared: of the tile's two chunks, loaded before its accumulator
                         // is waited for

  __device__ __forceinline__ Drain(const PairArgs& g, uint8_t* stage, __nv_bfloat16* bias,
                                   uint32_t res_bar, int grp, int r)
      : g(g), stage(stage), sw(r & 7), grp(grp), res_bar(res_bar), row_at(r * 128),
        first(r == 0), bias(bias) {}

  // The bias of 64 columns from `col` and of 64 from col + 128, in the tile's half `at` of the
  // place (the group's next barrier is before their use).
  __device__ __forceinline__ void load_bias(int at, int64_t col) const {
    const int r = row_at / 128;
    const int64_t c = col + (r >> 6) * 128 + (r & 63);
    if (g.ep.bias) bias[at * 128 + r] = c < g.N ? g.ep.bias[c] : __float2bfloat16_rn(0.0f);
  }
  __device__ __forceinline__ uint4* mine(int b) const {
    return reinterpret_cast<uint4*>(stage + b * kOutBytes + row_at);
  }
  __device__ __forceinline__ uint32_t addr(int b) const {
    return smem_u32(stage + b * kOutBytes);
  }

  // A buffer for the next chunk (with pre, which goes out first, both), and its residual: the
  // box that finish() stores to, and no other, since out may be the residual's buffer.
  __device__ __forceinline__ void open(const CUtensorMap& tm_res, int64_t col, int64_t row0) {
    if (first) {
      if (g.ep.pre)
        bulk_wait_read<0>();
      else
        bulk_wait_read<1>();
      if (ok && g.ep.residual && g.splits == 1) {
        mbar_arrive_expect_tx(res_bar, kOutBytes);
        tma_load_2d(addr(buf), &tm_res, res_bar, (int32_t)col, (int32_t)row0);
      }
    }
    group_sync(grp);
  }

  __device__ __forceinline__ void partial(const CUtensorMap& tm_out, const uint32_t (&v)[64],
                                          int64_t col, int64_t row0, unsigned split) {
    uint4* m = mine(buf);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      m[i ^ sw] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    fence_proxy_async_smem();
    group_sync(grp);
    if (first) {
      tma_store_3d(&tm_out, addr(buf), (int32_t)col, (int32_t)row0, (int32_t)split);
      bulk_commit();
    }
    buf ^= 1;
  }

  __device__ __forceinline__ void finish(const CUtensorMap& tm_out, const CUtensorMap& tm_pre,
                                         uint32_t (&v)[64], int64_t col, int64_t row0, int chunk) {
    if (g.ep.bias) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float bv[8];
        unpack8(reinterpret_cast<const uint4*>(bias + chunk * 64)[i], bv);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[8 * i + k] = __float_as_uint(__uint_as_float(v[8 * i + k]) + bv[k]);
      }
    }
    if (g.ep.pre) {
      uint4* m = mine(buf ^ 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i ^ sw] = pack8_bits(v + 8 * i);
      fence_proxy_async_smem();
      group_sync(grp);
      if (first) {
        tma_store_2d(&tm_pre, addr(buf ^ 1), (int32_t)col, (int32_t)row0);
        bulk_commit();
      }
    }
    if (g.ep.act != JM_ACT_NONE) apply_act(v, g.ep.act);
    if (g.ep.residual) {
      ok = ok && mbar_wait(res_bar, res_parity, g.err, 85);
      res_parity ^= 1u;
    }
    uint4* m = mine(buf);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (g.ep.residual) {
        float rv[8];
        unpack8(m[i ^ sw], rv);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[8 * i + k] = __float_as_uint(__uint_as_float(v[8 * i + k]) + rv[k]);
      }
      m[i ^ sw] = pack8_bits(v + 8 * i);
    }
    fence_proxy_async_smem();
    group_sync(grp);
    if (first) {
      tma_store_2d(&tm_out, addr(buf), (int32_t)col, (int32_t)row0);
      bulk_commit();
    }
    buf ^= 1;
  }

  __device__ __forceinline__ void close() const {
    if (first) bulk_wait_all();
  }
};

template <bool AMN, bool BMN, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ CUtensorMap tm_out,
                  const __grid_constant__ CUtensorMap tm_res,
                  const __grid_constant__ CUtensorMap tm_pre, const PairArgs g) {
  constexpr int kStage = stage_bytes(BN), kBHalf = BN / 2;
  const int S = stages(BN, g.single, g.cpairs > 1);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) __nv_bfloat16 bias_of[2][256];   // [group][tile parity][chunk][64]
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = g.single ? smem : smem + S * kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRegion);
  uint64_t* full = bars;              // [S] (leader) both CTAs' halves landed
  uint64_t* empty = full + kMaxStages;  // [S] the pair's MMAs have read the stage
  uint64_t* acc_full = empty + kMaxStages;  // [2] accumulator complete
  uint64_t* acc_empty = acc_full + 2; // [2] (leader) both epilogues are done (16 warps)
  uint64_t* res_full = acc_empty + 2; // [2] a group's residual box landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank(), rank = crank & 1;   // rank in the pair
  const bool leader = rank == 0;
  // (pairs of one cluster share a tile, and then a cluster has one)
  const unsigned pair = blockIdx.x / (2 * g.cpairs), npairs = gridDim.x / (2 * g.cpairs);
  const unsigned items = g.m_tiles * g.n_tiles * g.splits;
  const int kchunks = (int)((g.K + kK - 1) / kK);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 16);
      mbar_init(smem_u32(&res_full[b]), 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_b);
    prefetch_tmap(&tm_out);
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers exist before either signals the other's
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (before the wait: its divisions are 0.5 us of the first load's way)
  Item first{};
  if (warp == 0) first = item_of(g, pair, kchunks);
  if (!g.late_wait) grid_dep_wait();
  grid_dep_launch();
  // (a wait gives up after 2 s: no CTA can have recorded one yet)
  if (g.clear_err && blockIdx.x == 0 && threadIdx.x < sizeof(ErrFlags) / 4)
    reinterpret_cast<unsigned*>(g.err)[threadIdx.x] = 0u;

  if (warp == 0) {
    if (elect_one()) {
      Place at(S);
      bool ok = true;
      const uint32_t fb0 = cluster_addr(smem_u32(full), crank & ~1u), base = smem_u32(smem);
      for (unsigned w = pair; ok && w < items; w += npairs) {
        const Item q = w == pair ? first : item_of(g, w, kchunks);
        const int32_t m0 = (int32_t)(q.mt * (2 * kHalf) + rank * kHalf);
        const int32_t n0 = (int32_t)(q.nt * BN + rank * kBHalf);
        for (int kc = q.k0; kc < q.k1; ++kc, at.next()) {
          const int s = at.s;   // (the first round's wait for "empty" returns at once)
          if (!mbar_wait(smem_u32(&empty[s]), at.parity ^ 1u, g.err, 81)) {
            ok = false;
            break;
          }
          const uint32_t st = base + (uint32_t)(s * kStage), fb = fb0 + (uint32_t)(s * 8);
          // the leader expects both CTAs' bytes on its barrier
          if (leader) mbar_arrive_expect_tx(smem_u32(&full[s]), (uint32_t)(2 * kStage));
          if constexpr (AMN) {   // boxes of 64 m values x 64 k rows
            tma_load_2d_pair(st, &tm_a, fb, m0, kc * kK);
            tma_load_2d_pair(st + kABytes / 2, &tm_a, fb, m0 + 64, kc * kK);
          } else {
            tma_load_2d_pair(st, &tm_a, fb, kc * kK, m0);
          }
          if constexpr (BMN) {
#pragma unroll
            for (int h = 0; h < kBHalf / 64; ++h)
              tma_load_2d_pair(st + kABytes + h * 8192, &tm_b, fb, n0 + 64 * h, kc * kK);
          } else {
            tma_load_2d_pair(st + kABytes, &tm_b, fb, kc * kK, n0);
          }
        }
      }
      // The stages' last signals come from the pair's leader and are waited for here, so that
      // none is on its way to a CTA that has left.
      for (int i = 0; ok && i < S; ++i, at.next())
        ok = mbar_wait(smem_u32(&empty[at.s]), at.parity ^ 1u, g.err, 79);
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {
      const uint32_t idesc = idesc_bf16_f32_major(2 * kHalf, BN, AMN, BMN);
      const uint16_t both = (uint16_t)(0x3u << crank);   // the pair's CTAs (crank is even here)
      Place at(S);
      Place acc(2);
      bool ok = true;
      const uint32_t base = smem_u32(smem);
      const uint64_t ad_base = AMN ? sw128_mnmajor_desc(base, 8192) : sw128_kmajor_desc(base);
      const uint64_t bd_base = BMN ? sw128_mnmajor_desc(base + kABytes, 8192)
                                   : sw128_kmajor_desc(base + kABytes);
      for (unsigned w = pair; ok && w < items; w += npairs, acc.next()) {
        const Item q = item_of(g, w, kchunks);
        const int b = acc.s;
        if (!mbar_wait(smem_u32(&acc_empty[b]), acc.parity ^ 1u, g.err, 82)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)(b * 256);
        for (int kc = q.k0; kc < q.k1; ++kc, at.next()) {
          const int s = at.s;
          if (!mbar_wait(smem_u32(&full[s]), at.parity, g.err, 83)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // descriptors by addition: the start address is their low 14 bits, in 16 bytes
          const uint64_t ad0 = ad_base + (uint64_t)(s * (kStage / 16));
          const uint64_t bd0 = bd_base + (uint64_t)(s * (kStage / 16));
#pragma unroll
          for (int kk = 0; kk < kK / 16; ++kk)
            umma_f16_pair(d_tmem, ad0 + kk * (AMN ? 128 : 2), bd0 + kk * (BMN ? 128 : 2), idesc,
                          (kc > q.k0 || kk > 0) ? 1u : 0u);
          umma_commit_pair(smem_u32(&empty[s]), both);
        }
        if (ok) umma_commit_pair(smem_u32(&acc_full[b]), both);
      }
      // The pair's other CTA signals acc_empty by arrives that nothing orders before the last
      // cluster barrier: this CTA may not leave before those of its last two tiles are in.
      // (A cluster that shares a tile never signals it.)
      for (int i = 0; ok && g.cpairs == 1 && i < 2; ++i, acc.next())
        ok = mbar_wait(smem_u32(&acc_empty[acc.s]), acc.parity ^ 1u, g.err, 78);
    }
  } else {
    // epilogue: this CTA's 128 rows of the pair's 256-row tile, a row per thread; two
    // groups of 4 warps take the 128-byte column chunks in turn
    const int lg = warp & 3, grp = (warp - 2) >> 2, r = lg * 32 + lane;
    const bool split = g.splits > 1;
    const int cw = split ? 32 : 64;                   // columns in 128 bytes
    const uint32_t acc_empty_leader = cluster_addr(smem_u32(&acc_empty[0]), crank & ~1u);
    Drain d(g, staging + grp * 2 * kOutBytes, bias_of[grp], smem_u32(&res_full[grp]), grp, r);
    // (a thread whose wait ran out goes on without waiting, so that its group's barriers
    // stay matched; the error header says that the values are not to be used)
    if (g.cpairs > 1) {
      // One tile; the half of its columns that this pair finishes, a chunk of 64 a group
      // (128 wide: of the first one alone).
      constexpr int kCols = BN / 2;
      const Item q = item_of(g, pair, kchunks);
      const int64_t row0 = (int64_t)q.mt * (2 * kHalf) + rank * kHalf, n0 = (int64_t)q.nt * BN;
      const int own = (int)(crank >> 1) * kCols + grp * 64, theirs = (int)(~crank >> 1 & 1) * kCols;
      const int64_t col = n0 + own;
      const bool rows = row0 < g.M, mine = rows && grp * 64 < kCols && col < g.N;
      const uint32_t tbase = tmem + ((uint32_t)(lg * 32) << 16);
      // 4 columns of all rows after one another, so that rows are 16 bytes apart
      const float4* joined = reinterpret_cast<float4*>(smem + kRegion - joined_bytes(BN)) + r;
      if (mine) d.load_bias(0, col);
      d.ok = mbar_wait(smem_u32(&acc_full[0]), 0, g.err, 84);
      tc_fence_after();
      if (mine) d.open(tm_res, col, row0);
      if (rows) {
        const uint32_t to = cluster_addr(smem_u32(joined), crank ^ 2u);
        for (int c = grp * (kCols / 2); c < (grp + 1) * (kCols / 2); c += 32) {
          uint32_t v[32];
          tmem_ld16(tbase + theirs + c, *reinterpret_cast<uint32_t(*)[16]>(v));
          tmem_ld16(tbase + theirs + c + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            st_cluster4(to + (uint32_t)((c / 4 + i) * kHalf * 16), v[4 * i], v[4 * i + 1],
                        v[4 * i + 2], v[4 * i + 3]);
        }
      }
      cluster_sync();   // (warps 0 and 1 come to it below)
      if (mine) {
        uint32_t v[64];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tmem_ld16(tbase + own + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(v + 16 * i));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 f = joined[(grp * 16 + i) * kHalf];
          const float o[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[4 * i + k] = __float_as_uint(__uint_as_float(v[4 * i + k]) + o[k]);
        }
        d.finish(tm_out, tm_pre, v, col, row0, 0);
      }
      d.close();
    }
    Place acc(2);
    for (unsigned w = pair; g.cpairs == 1 && w < items; w += npairs, acc.next()) {
      const Item q = item_of(g, w, kchunks);
      const int b = acc.s;
      const int64_t row0 = (int64_t)q.mt * (2 * kHalf) + rank * kHalf, n0 = (int64_t)q.nt * BN;
      const bool rows = row0 < g.M;
      const uint32_t tbase = tmem + ((uint32_t)(lg * 32) << 16) + (uint32_t)(b * 256);
      bool waited = false;
      if (!split) d.load_bias(b, n0 + grp * 64);
      for (int c = grp * cw; rows && c < BN && n0 + c < g.N; c += 2 * cw) {
        const int64_t col = n0 + c;
        if (!g.single) d.open(tm_res, col, row0);
        if (!waited) d.ok = d.ok && mbar_wait(smem_u32(&acc_full[b]), acc.parity, g.err, 84);
        waited = true;
        if (g.single) d.open(tm_res, col, row0);   // the staging was the ring's until now
        tc_fence_after();
        uint32_t v[64];
        tmem_ld16(tbase + c, *reinterpret_cast<uint32_t(*)[16]>(v));
        tmem_ld16(tbase + c + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
        if (split) {
          tmem_ld_wait();
          d.partial(tm_out, v, col, row0, q.split);
        } else {
          tmem_ld16(tbase + c + 32, *reinterpret_cast<uint32_t(*)[16]>(v + 32));
          tmem_ld16(tbase + c + 48, *reinterpret_cast<uint32_t(*)[16]>(v + 48));
          tmem_ld_wait();
          d.finish(tm_out, tm_pre, v, col, row0, 2 * b + (c >> 7));
        }
      }
      // the accumulator is free once it is complete and this warp has read its part
      if (!waited) d.ok = d.ok && mbar_wait(smem_u32(&acc_full[b]), acc.parity, g.err, 84);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_leader + (uint32_t)(b * 8));
    }
    if (g.cpairs == 1) d.close();
  }
  if (g.cpairs > 1 && warp < 2) {
    __syncwarp();
    cluster_sync();   // the cluster's halves are there
  }
  if (g.late_wait) grid_dep_wait();
  tc_fence_before();
  // No CTA leaves while another may still signal it.  The barrier itself orders no signal;
  // each is waited for by the CTA it goes to: full by the MMAs, acc_full by the epilogue,
  // empty by the producer and acc_empty by the leader's MMA warp at their ends.
  cluster_sync_relaxed();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// The partial tiles of a K split, added in split order, then the epilogue.
__global__ void __launch_bounds__(256)
    k_linear_reduce(const float* __restrict__ part, int splits, int64_t M, int64_t N,
                    const Epilogue ep) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t n8 = N / 8, total = M * n8;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / n8, col = (i - row * n8) * 8, at = row * N + col;
    float v[8] = {};
    for (int s = 0; s < splits; ++s) {
      const float4* p = reinterpret_cast<const float4*>(part + (int64_t)s * M * N + at);
      const float4 a = __ldcs(p), b = __ldcs(p + 1);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    finish8(ep, v, at, col);
  }
}

// g_p = g_out act'(pre) in bf16 (the operand of both products) and, for g_bias, its
// column sums (unrounded, float32) over this CTA's rows.  A CTA takes 8 tx columns (8 per
// thread) x `rows` rows, 256 / tx of them at a time, so that a narrow matrix keeps its
// threads busy too; one read of g_out and pre, one write of g_p.
constexpr int kGpThreads = 256;

__global__ void __launch_bounds__(kGpThreads)
    k_linear_gpre(const __nv_bfloat16* __restrict__ g_out, const __nv_bfloat16* __restrict__ pre,
                  int act, int64_t M, int64_t N, int tx, int rows, __nv_bfloat16* __restrict__ gp,
                  float* __restrict__ part, ErrFlags* err) {
  __shared__ float sums[kGpThreads * 8];   // [256 / tx][8 tx]
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < sizeof(ErrFlags) / 4)
    reinterpret_cast<unsigned*>(err)[threadIdx.x] = 0u;
  const int x = threadIdx.x & (tx - 1), y = threadIdx.x / tx, step = kGpThreads / tx;
  const int64_t col0 = (int64_t)blockIdx.x * tx * 8, col = col0 + x * 8;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = min(M, r0 + rows);
  float sum[8] = {};
  if (col < N) {
#pragma unroll 4
    for (int64_t r = r0 + y; r < r1; r += step) {
      float g[8];
      unpack8(*reinterpret_cast<const uint4*>(g_out + r * N + col), g);
      if (pre) {
        float p[8];
        unpack8(*reinterpret_cast<const uint4*>(pre + r * N + col), p);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= act_grad(p[j], act);
        *reinterpret_cast<uint4*>(gp + r * N + col) = pack8(g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += g[j];
    }
  }
  if (!part) return;
  float4* d = reinterpret_cast<float4*>(step > 1 ? sums + threadIdx.x * 8
                                                 : part + (int64_t)blockIdx.y * N + col);
  if (step > 1 || col < N) {
    d[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    d[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
  }
  if (step == 1) return;   // (uniform in the CTA)
  __syncthreads();
  for (int c = threadIdx.x; c < tx * 8 && col0 + c < N; c += kGpThreads) {
    float acc = 0.0f;
    for (int q = 0; q < step; ++q) acc += sums[q * tx * 8 + c];
    part[(int64_t)blockIdx.y * N + col0 + c] = acc;
  }
}

// Column sums of the partial rows in a fixed order (32 interleaved chains).
__global__ void __launch_bounds__(1024)
    k_linear_bias_reduce(const float* __restrict__ part, int64_t rows, int64_t N,
                         __nv_bfloat16* __restrict__ g_bias) {
  __shared__ float sh[32][33];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float acc = 0.0f;
  if (c < N)
#pragma unroll 4
    for (int64_t r = threadIdx.y; r < rows; r += 32) acc += part[r * N + c];
  sh[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.y == 0 && c < N) {
#pragma unroll
    for (int i = 1; i < 32; ++i) acc += sh[i][threadIdx.x];
    g_bias[c] = __float2bfloat16_rn(acc);
  }
}

// ------------------------------------------------------------------ host side

// A row-major bf16 matrix [outer][inner] as boxes of 64 inner values x `box` rows.
bool bf16_map(CUtensorMap* m, const void* base, int64_t outer, int64_t inner, int box) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)inner * 2};
  cuuint32_t bx[2] = {(cuuint32_t)kK, (cuuint32_t)box}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Partial tiles [splits][M][N], float32, as boxes of 32 columns x 128 rows.
bool part_map(CUtensorMap* m, const void* base, int64_t splits, int64_t M, int64_t N) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)M, (cuuint64_t)splits};
  cuuint64_t strides[2] = {(cuuint64_t)N * 4, (cuuint64_t)(M * N) * 4};
  cuuint32_t bx[3] = {32, kHalf, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kPairs = 74;   // CTA pairs of a B200 (148 SMs)

// How a product is cut: tile width, pairs of a cluster on a tile, K splits through memory.
struct Cut {
  int bn, cpairs, splits;
};

// Estimated microseconds, without the start and the end that every cut has alike (some 5 us):
// waves of work items on 74 pairs (a 64-wide chunk of a 256 x 256 tile takes a pair 0.28 us, of a
// 256 x 128 tile 0.16); 1 us for a cluster's exchange; for splits the partial tiles' round trip
// through L2 and one launch.  Each product is cut by itself.  Measured:
// 256 x 8192 x 4096 two pairs 20 us, two splits 23; 530 x 5496 x 2208 one wave of two pairs a
// 256 x 256 tile 23.5 us, of uncut 256 x 128 tiles 28.7; 600 x 2048 x 512 two pairs
// 7.3 us, 4 splits 8.0, uncut 9.2.  (Tiles of 4 pairs took 6 us more than their splits.)
Cut choose_cut(int64_t M, int64_t N, int64_t K) {
  const int64_t chunks = (K + kK - 1) / kK;
  Cut best{256, 1, 1};
  double best_us = 1e30;
  for (int bn = 256; bn >= 128; bn /= 2) {
    const int64_t tiles = ((M + 255) / 256) * ((N + bn - 1) / bn);
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && chunks / s < 2) break;
      const int64_t waves = (tiles * s + kPairs - 1) / kPairs;
      const double us = (double)(waves * ((chunks + s - 1) / s)) * (bn == 256 ? 0.28 : 0.16);
      // (a B200 holds 33 clusters of 4 CTAs with one CTA an SM)
      if (s == 1 || (s == 2 && tiles <= 33)) {
        const double c = us + (s == 1 ? 0.0 : 1.0);
        if (c < best_us * 0.999) {
          best_us = c;
          best = {bn, s, 1};
        }
      }
      if (s > 1) {
        const double m = us + 1.5 + (double)M * (double)N * 4.0 * (2 * s + 1) / 6.0e6;
        if (m < best_us * 0.999) {
          best_us = m;
          best = {bn, 1, s};
        }
      }
    }
  }
  return best;
}

size_t part_bytes(int64_t M, int64_t N, int64_t K) {
  const Cut c = choose_cut(M, N, K);
  return c.splits > 1 ? align256((size_t)c.splits * M * N * 4) : 0;
}

int cached_attr(std::atomic<int>* cache, int dev, int (*query)()) {
  if (dev < 0 || dev >= 64) return query();
  int v = cache[dev].load(std::memory_order_relaxed);
  if (!v) cache[dev].store(v = query(), std::memory_order_relaxed);
  return v;
}

template <bool AMN, bool BMN, int BN>
int query_pairs() {
  auto kern = k_linear_pair<AMN, BMN, BN>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
      cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * kPairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
  return n;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster,
                   cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool AMN, bool BMN, int BN>
cudaError_t launch_pair(const CUtensorMap (&tm)[5], const PairArgs& g, cudaStream_t s) {
  static std::atomic<int> cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int most = cached_attr(cache, dev, query_pairs<AMN, BMN, BN>);
  if (most <= 0) return cudaErrorInvalidConfiguration;
  const int64_t items = (int64_t)g.m_tiles * g.n_tiles * g.splits;
  const int64_t clusters = g.single || items < most ? items : most;
  return launch(k_linear_pair<AMN, BMN, BN>, dim3((unsigned)(2 * g.cpairs * clusters)),
                dim3(kThreads), (size_t)kSmemBytes, 2 * g.cpairs, s, tm[0], tm[1], tm[2], tm[3], tm[4], g);
}

// C[M, N] = A . B^T with the epilogue `ep`.  AMN / BMN: A is stored [K, M], B [K, N].
// `apart`: see late_wait.
template <bool AMN, bool BMN>
cudaError_t product(int64_t M, int64_t N, int64_t K, const void* A, const void* B,
                    const Epilogue& ep, float* part, ErrFlags* err, bool clear_err, bool apart, Problem& p) {
  const Cut c = choose_cut(M, N, K);
  CUtensorMap tm[5];
  bool ok = (AMN ? bf16_map(&tm[0], A, K, M, 64) : bf16_map(&tm[0], A, M, K, kHalf)) &&
            (BMN ? bf16_map(&tm[1], B, K, N, 64) : bf16_map(&tm[1], B, N, K, c.bn / 2)) &&
            (c.splits > 1 ? part_map(&tm[2], part, c.splits, M, N)
                          : bf16_map(&tm[2], ep.out, M, N, kHalf));
  tm[3] = tm[4] = tm[2];
  if (ep.residual) ok = ok && bf16_map(&tm[3], ep.residual, M, N, kHalf);
  if (ep.pre) ok = ok && bf16_map(&tm[4], ep.pre, M, N, kHalf);
  if (!ok) return cudaErrorInvalidValue;
  PairArgs g{};
  g.M = M;
  g.N = N;
  g.K = K;
  g.m_tiles = (unsigned)((M + 255) / 256);
  g.n_tiles = (unsigned)((N + c.bn - 1) / c.bn);
  g.cpairs = c.cpairs;
  g.splits = c.splits;
  g.ep = ep;
  g.err = err;
  g.single = (int64_t)g.m_tiles * g.n_tiles * g.splits <= kPairs || c.cpairs > 1;
  g.clear_err = clear_err;
  g.late_wait = apart && !clear_err && c.splits == 1;   // (the partial tiles' place is shared)
  cudaError_t e = c.bn == 256 ? launch_pair<AMN, BMN, 256>(tm, g, p.stream)
                              : launch_pair<AMN, BMN, 128>(tm, g, p.stream);
  if (e != cudaSuccess) return e;
  launched(p, "k_linear_pair");
  if (c.splits > 1) {
    const int64_t n = M * N / 8;
    const int64_t ctas = (n + 255) / 256 < 148 * 8 ? (n + 255) / 256 : 148 * 8;
    e = launch(k_linear_reduce, dim3((unsigned)ctas), dim3(256), 0, 1, p.stream, (const float*)part,
               c.splits, M, N, ep);
    if (e == cudaSuccess) launched(p, "k_linear_reduce");
  }
  return e;
}

// Threads of a CTA of k_linear_gpre along the columns (a power of two), and rows a CTA
// takes: enough CTAs for the GPU, at least 4 rows a thread.
int gpre_tx(int64_t N) {
  // the widest that leaves fewest columns behind the matrix's end, down to 512 bytes a row
  // (the whole backward at 4847 x 64 -> 2440, whose second column of CTAs was 81% idle at 256,
  // and with cuts of its products: 60 -> 45 us)
  int best = 32;
  double most = 0.0;
  for (int tx = kGpThreads; tx >= 32; tx /= 2) {
    const double used = (double)N / (double)((N + tx * 8 - 1) / (tx * 8) * (tx * 8));
    if (used > most * 1.05) {
      most = used;
      best = tx;
    }
  }
  while (best > 8 && best * 4 >= N) best /= 2;   // a narrow matrix
  return best;
}

int gpre_rows(int64_t M, int64_t N) {
  const int tx = gpre_tx(N);
  const int64_t col_ctas = (N + tx * 8 - 1) / (tx * 8), least = 4 * (kGpThreads / tx);
  // one wave of 5 CTAs an SM
  const int64_t row_ctas = col_ctas < 148 * 5 ? 148 * 5 / col_ctas : 1;
  int64_t r = (M + row_ctas - 1) / row_ctas;
  r = r < least ? least : r;
  if (r < (M + 65534) / 65535) r = (M + 65534) / 65535;   // grid y limit
  return (int)r;
}

// Backward workspace: [header][g_p bf16][bias partial rows][partial tiles of the
// larger split product].
struct BwdWs {
  __nv_bfloat16* gp;
  float* bias_part;
  float* part;
  size_t bytes;
};

BwdWs bwd_ws(int64_t M, int64_t K, int64_t N, int act, char* base) {
  BwdWs w{};
  size_t off = sizeof(ErrFlags);
  auto take = [&](size_t n) {
    char* p = base ? base + off : nullptr;
    off += align256(n);
    return p;
  };
  w.gp = reinterpret_cast<__nv_bfloat16*>(take(act == JM_ACT_NONE ? 0 : (size_t)M * N * 2));
  const int64_t rows = M ? (M + gpre_rows(M, N) - 1) / gpre_rows(M, N) : 0;
  w.bias_part = reinterpret_cast<float*>(take((size_t)rows * N * 4));
  const size_t px = M && !linear_few(M, N) ? part_bytes(M, K, N) : 0, pw = M ? part_bytes(N, K, M) : 0;
  w.part = reinterpret_cast<float*>(take(px > pw ? px : pw));
  w.bytes = off;
  return w;
}

}  // namespace

size_t linear_fwd_ws_bytes(int64_t M, int64_t K, int64_t N) {
  return sizeof(ErrFlags) + (M && !linear_few(M, K) ? part_bytes(M, N, K) : 0);
}

size_t linear_bwd_ws_bytes(int64_t M, int64_t K, int64_t N, int act) {
  return bwd_ws(M, K, N, act, nullptr).bytes;
}

cudaError_t run_linear_fwd(const LinearArgs& a, Problem& p) {
  ErrFlags* err = reinterpret_cast<ErrFlags*>(a.ws);
  if (a.M == 0) return cudaMemsetAsync(err, 0, sizeof(ErrFlags), p.stream);
  Epilogue ep{};
  ep.bias = static_cast<const __nv_bfloat16*>(a.bias);
  ep.residual = static_cast<const __nv_bfloat16*>(a.residual);
  ep.out = static_cast<__nv_bfloat16*>(a.out);
  ep.pre = static_cast<__nv_bfloat16*>(a.pre);
  ep.act = a.act;
  launches_begin(p);
  if (linear_few(a.M, a.K))
    return run_linear_few(a.M, a.N, a.K, a.x, a.w, false, ep, err, true, false, p);
  return product<false, false>(a.M, a.N, a.K, a.x, a.w, ep,
                               reinterpret_cast<float*>(a.ws + sizeof(ErrFlags)), err, true, false, p);
}

cudaError_t run_linear_bwd(const LinearArgs& a, Problem& p) {
  ErrFlags* err = reinterpret_cast<ErrFlags*>(a.ws);
  if (a.M == 0) {  // nothing flows back: the sums over rows are zero
    cudaError_t e = cudaMemsetAsync(err, 0, sizeof(ErrFlags), p.stream);
    if (e == cudaSuccess && a.g_w) e = cudaMemsetAsync(a.g_w, 0, (size_t)a.N * a.K * 2, p.stream);
    if (e == cudaSuccess && a.g_bias) e = cudaMemsetAsync(a.g_bias, 0, (size_t)a.N * 2, p.stream);
    return e;
  }
  const BwdWs w = bwd_ws(a.M, a.K, a.N, a.act, a.ws);
  const void* gp = a.g_out;
  cudaError_t e = cudaSuccess;
  launches_begin(p);
  const bool grad = a.act != JM_ACT_NONE && (a.g_x || a.g_w || a.g_bias);
  if (grad || a.g_bias) {
    const int rows = gpre_rows(a.M, a.N);
    const int tx = gpre_tx(a.N);
    const dim3 grid((unsigned)((a.N + tx * 8 - 1) / (tx * 8)), (unsigned)((a.M + rows - 1) / rows));
    e = launch(k_linear_gpre, grid, dim3(kGpThreads), 0, 1, p.stream,
               static_cast<const __nv_bfloat16*>(a.g_out),
               grad ? static_cast<const __nv_bfloat16*>(a.pre) : nullptr, a.act, a.M, a.N, tx, rows,
               w.gp, a.g_bias ? w.bias_part : nullptr, err);
    if (e != cudaSuccess) return e;
    launched(p, "k_linear_gpre");
    if (grad) gp = w.gp;
    if (a.g_bias) {
      e = launch(k_linear_bias_reduce, dim3((unsigned)((a.N + 31) / 32)), dim3(32, 32), 0, 1, p.stream,
                 (const float*)w.bias_part, (int64_t)grid.y, a.N,
                 static_cast<__nv_bfloat16*>(a.g_bias));
      if (e != cudaSuccess) return e;
      launched(p, "k_linear_bias_reduce");
    }
  } else if (!a.g_x && !a.g_w) {
    return cudaMemsetAsync(err, 0, sizeof(ErrFlags), p.stream);
  }
  const bool clear = !grad && !a.g_bias;   // else k_linear_gpre has done it
  Epilogue ep{};
  ep.act = JM_ACT_NONE;
  if (a.g_x) {  // [M, K] = g_p [M, N] . w [N, K]
    ep.out = static_cast<__nv_bfloat16*>(a.g_x);
    // (apart from the bias's sums where these came last)
    e = linear_few(a.M, a.N)
            ? run_linear_few(a.M, a.K, a.N, gp, a.w, true, ep, err, clear, a.g_bias != nullptr, p)
            : product<false, true>(a.M, a.K, a.N, gp, a.w, ep, w.part, err, clear,
                                   a.g_bias != nullptr, p);
    if (e != cudaSuccess) return e;
  }
  if (a.g_w) {  // [N, K] = g_p [M, N]^T . x [M, K]
    ep.out = static_cast<__nv_bfloat16*>(a.g_w);
    e = product<true, true>(a.N, a.K, a.M, gp, a.x, ep, w.part, err, clear && !a.g_x,
                            a.g_x || a.g_bias, p);
  }
  return e;
}

}  // namespace jmix
