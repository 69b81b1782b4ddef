// A whole mixture-of-experts layer for few tokens in two kernels.
//
//   logits = x Wr^T;  the top_k experts of each token (softmax weights g)
//   h   = silu(x Wgate_e^T) (x Wup_e^T)     for each (token, chosen expert) pair
//   out = sum_i g_i h_i Wdown_{e_i}^T + residual
//
// k_moe_route: one CTA, or with few tokens a cluster, per token; logits, choice, weights.
// k_moe: one CTA per SM streams the chosen experts' weights, once for each block of an
// expert's tokens (moe_block: 16 to 128 rows, twice an even router's share).  With few tokens
// those bytes bound the layer (an expert of 4096 x 14336 is 352 MB: 54 us of HBM time,
// its products for 32 tokens 7 us of tensor time), so the design keeps HBM busy:
//
// * The weights are the MMA's A operand (128 rows of weights = TMEM lanes), the tokens
//   its N: few tokens waste tensor time that is free here, and no weight is read twice for a
//   block.  An expert that gets more rows than one block holds is streamed again for the next
//   one.  256 tokens of 4096, floors behind the times: one expert of 14336, two blocks, 127 us,
//   54; 16 experts, top 2, the same two chosen by every token, four blocks each, 354 us, 107.
// * A phase's work is a line of units (block of an expert's tokens, tile of weight rows)
//   x K steps of 64, cut into equal contiguous ranges, one per CTA: every SM streams the
//   same bytes whatever the number of blocks.  A step brings 256 weight rows:
//   128 of gate and the same 128 of up in the first phase (so that h is formed in the
//   thread that holds both), 256 of down in the second.
// * A unit inside one CTA's range is finished from TMEM.  A cut one leaves float32
//   partial tiles, each CTA of it then finishing its share of the columns; partial tiles
//   are added in CTA order, so results do not depend on timing.
// * Warp 0 streams weights, warps 6 and 7 half of the tokens' rows each (gathered by index 4
//   at a time, some 45 cycles of one thread, then rows of h), warp 1 issues the MMAs, warps
//   2-5 drain them.  Nothing but warps 6 and 7 waits between the phases, and only for h of
//   the block they need, so the ring is full of down-projection weights when h arrives.
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

constexpr int kThreads = 256;
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

// Routing lists, rebuilt by every CTA in shared memory, of the call's sizes (what they do not
// take is the ring's).  Pair rows (token, choice) are sorted by expert, tokens ascending.
struct Lists {
  Entry* entry;
  int* count;        // [E]
  int* first;        // [E] first pair row of an expert
  int* n_entries;
  uint16_t* token;   // [P] of a pair row
  uint16_t* ent;     // [P] block of a pair row
  uint16_t* row;     // [P] pair row of token * top_k + choice
  uint16_t* block;   // [E] first block of an expert
  __device__ __forceinline__ Lists(uint8_t* at, int P, int E, int NB) {
    entry = reinterpret_cast<Entry*>(at);
    count = reinterpret_cast<int*>(entry + most_entries(P, E, NB));
    first = count + E;
    n_entries = first + E;
    token = reinterpret_cast<uint16_t*>(n_entries + 1);
    ent = token + P;
    row = ent + P;
    block = row + P;
  }
  // every expert's last block, and the full ones before them
  static __host__ __device__ int most_entries(int P, int E, int NB) {
    return (E < P ? E : P) + P / NB;
  }
  static size_t bytes(int P, int E, int NB) {
    const size_t n = sizeof(Entry) * most_entries(P, E, NB) + 4 * (2 * (size_t)E + 1) +
                     2 * (3 * (size_t)P + E);
    return (n + 255) / 256 * 256;
  }
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

// A phase's line of work: units of `ksteps` steps in `ppu` parts of `quant` steps (the last
// one may have fewer), the parts cut between `ctas` CTAs.
struct Line {
  unsigned tiles, ksteps, quant, ppu, parts, ctas;
  unsigned base, rest;   // parts = base ctas + rest
  float inv_ctas;
  double inv;            // 1 / parts
  // the first part of CTA c's range: floor(c parts / ctas).  (c rest is below 2^16 and the
  // quotient's distance from an integer at least 0.5 / 160: float32 is exact.)
  __device__ __forceinline__ unsigned first_part(unsigned c) const {
    c = min(c, ctas);
    return c * base + (unsigned)(((float)(c * rest) + 0.5f) * inv_ctas);
  }
  // the CTA whose range holds the part p: ((p + 1) ctas - 1) / parts (below 2^32, checked
  // on the host; by a multiplication, which may be one off)
  __device__ __forceinline__ unsigned cta_of_part(unsigned p) const {
    const unsigned x = (p + 1) * ctas - 1;
    unsigned q = (unsigned)((double)x * inv);
    const int r = (int)(x - q * parts);
    if (r < 0) --q;
    if (r >= (int)parts) ++q;
    return q;
  }
  // the first and the last CTA of a unit
  __device__ __forceinline__ void ctas_of(unsigned unit, unsigned& c0, unsigned& c1) const {
    c0 = cta_of_part(unit * ppu);
    c1 = ppu == 1 ? c0 : cta_of_part((unit + 1) * ppu - 1);
  }
};

// Whole units or cut ones?  Cut ranges give every CTA the same bytes, but their partial
// tiles cost `join_us`.  Whole units leave the last round's CTAs to themselves, and one SM's
// loads from HBM reach about 60 GB/s: a step of 32 KB takes the whole GPU 5 ns, but one SM
// 550 ns.  Measured: one token, 2 of 16 experts of 4096 x 14336 (224 units of 64 steps), cut
// 128 us, whole 136 us; 13 tokens, 8 experts of 512 x 1416 (96 units of 8 steps), cut 34 us,
// whole 27 us.  Where ranges are short a unit is cut into at most `most` parts, since
// somebody has to add them all (2 units of 64 steps cut into single ones: 35 us).  There are
// no more CTAs than parts, so that no range between two others is empty.
__device__ __forceinline__ Line make_line(unsigned entries, unsigned rows, unsigned kdim,
                                          unsigned tile_rows, float join_us, unsigned log2_most) {
  Line l;
  l.tiles = (rows + tile_rows - 1) / tile_rows;
  l.ksteps = (kdim + kK - 1) / kK;
  const unsigned units = entries * l.tiles;
  const unsigned total = units * l.ksteps;
  const unsigned rounds = units / gridDim.x, rest = units - rounds * gridDim.x;
  const float all = (float)(rounds * gridDim.x * l.ksteps) * 0.005f, k = (float)l.ksteps;
  const float whole = fmaxf(all, (float)(rounds * l.ksteps) * 0.55f) +
                      (rest ? fmaxf((float)rest * k * 0.005f, k * 0.55f) : 0.0f);
  const unsigned least = (l.ksteps + (1u << log2_most) - 1) >> log2_most;   // steps of a part
  const float cut = fmaxf((float)total * 0.005f,
                          fmaxf((float)total / (float)gridDim.x, (float)least) * 0.55f);
  l.quant = whole <= cut + join_us          ? l.ksteps
            : total >= least * gridDim.x  ? 1u     // ranges of `least` steps by themselves
                                            : least;
  l.ppu = (l.ksteps + l.quant - 1) / l.quant;
  l.parts = units * l.ppu;
  l.ctas = max(min(gridDim.x, l.parts), 1u);
  l.base = l.parts / l.ctas;
  l.rest = l.parts - l.base * l.ctas;
  l.inv_ctas = 1.0f / (float)l.ctas;
  // (one Newton step from float32: a division in float64 would hold up the first loads)
  const double n = (double)max(l.parts, 1u), r = (double)(1.0f / (float)max(l.parts, 1u));
  l.inv = r * (2.0 - n * r);
  return l;
}

// A CTA's walk over its range of a line, unit by unit (divisions only at its start: with
// one or two in each step of the producing thread a step took it 550 ns).
struct Walk {
  unsigned s, s1, ent, tile, k, ksteps, tiles;
  Walk() = default;
  __device__ __forceinline__ explicit Walk(const Line& l) : ksteps(l.ksteps), tiles(l.tiles) {
    const unsigned p = l.first_part(blockIdx.x), p1 = l.first_part(blockIdx.x + 1);
    const unsigned u = p / l.ppu, u1 = p1 / l.ppu;
    k = (p - u * l.ppu) * l.quant;
    s = u * ksteps + k;
    s1 = u1 * ksteps + (p1 - u1 * l.ppu) * l.quant;
    ent = u / tiles;
    tile = u - ent * tiles;
  }
  __device__ __forceinline__ bool more() const { return s < s1; }
  // steps of the present unit in the range
  __device__ __forceinline__ unsigned steps() const { return min(s1 - s, ksteps - k); }
  __device__ __forceinline__ bool whole() const { return k == 0 && s1 - s >= ksteps; }
  __device__ __forceinline__ void next() {
    s += steps();
    k = 0;
    if (++tile == tiles) {
      tile = 0;
      ++ent;
    }
  }
};

// A place in a ring of n and the parity of its round.
struct Place {
  unsigned s = 0, parity = 0;
  __device__ __forceinline__ void skip(unsigned steps, unsigned n) {
    const unsigned to = s + steps, rounds = to / n;
    s = to - rounds * n;
    parity ^= rounds & 1u;
  }
  __device__ __forceinline__ void next(unsigned n) {
    if (++s == n) {
      s = 0;
      parity ^= 1u;
    }
  }
};

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

// Drain warps: whether `ok` holds in all of them.
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Drain warps: counts `v` after all of their earlier writes (the barrier orders them before
// the counting thread's release).
__device__ __forceinline__ void epi_add(unsigned* p, unsigned v, int et) {
  epi_sync();
  if (et == 0) add_release(p, v);
}

// One warp waits for a count.
__device__ __forceinline__ bool warp_wait(unsigned* p, unsigned n, ErrFlags* err, unsigned site) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_count(p, n, err, site) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
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

// A token's logits by a cluster of CTAs that share its experts (one CTA alone reads a
// router of 16 x 4096 in 10 us, most of it latency: with few tokens a cluster of 8 does).
// Products of bf16 are exact in float32 (inside its range) and added in float64, so that
// close logits keep their order: a choice that flips is a whole expert, not a last bit.  (With
// 8 of them added in float32 first, an x with one channel 30000 times the others mixed up
// logits 1e-5 apart.)  One conversion a product: 256 tokens of 4096, the layer with 16 experts
// of d_ff 64 37.4 us, with 256 experts 167 us; both factors converted 40.8 and 224 us; sums of
// 8 in float32 34.9 and 138 us.  The grid is [tokens][cluster].
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(const MoeKArgs a) {
  constexpr int kW = kRouteThreads / 32;
  __shared__ double logits[kMaxExperts];   // rank 0: of all experts
  __shared__ double slices[kMaxExperts > kW ? kMaxExperts : kW];
  const int t = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x, ranks = gridDim.x;
  cluster_sync();   // every CTA of the cluster runs before one writes to another
  grid_dep_wait();
  grid_dep_launch();
  if (t == 0 && rank == 0) {
    unsigned* s = reinterpret_cast<unsigned*>(a.sync);
    for (unsigned i = threadIdx.x; i < sizeof(Sync) / 4; i += kRouteThreads) s[i] = 0u;
    if (threadIdx.x < sizeof(ErrFlags) / 4) reinterpret_cast<unsigned*>(a.err)[threadIdx.x] = 0u;
  }
  // this CTA's experts rank, rank + ranks, ...; few of them are cut along D too, alike in
  // every CTA, so that equal rows of the router give equal logits
  const int mine = (a.E - rank + ranks - 1) / ranks, most = (a.E + ranks - 1) / ranks;
  int cuts = 1;
  while (most * cuts * 2 <= kW) cuts *= 2;
  const int n8 = a.D / 8;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x) + (int64_t)t * n8;
  for (int j = warp; j < mine * cuts; j += kW) {
    const int e = rank + j / cuts * ranks, cut = j % cuts;
    const uint4* wr = reinterpret_cast<const uint4*>(a.wr) + (int64_t)e * n8;
    double acc = 0.0, acc1 = 0.0;
#pragma unroll 8
    for (int i = cut * 32 + lane; i < n8; i += 32 * cuts) {
      float xv[8], wv[8];
      unpack8(xr[i], xv);
      unpack8(__ldg(wr + i), wv);
#pragma unroll
      for (int q = 0; q < 8; q += 2) {
        acc += (double)(xv[q] * wv[q]);
        acc1 += (double)(xv[q + 1] * wv[q + 1]);
      }
    }
    acc += acc1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) slices[j] = acc;
  }
  __syncthreads();
  const uint32_t to = leader_addr(smem_u32(logits));
  for (int j = threadIdx.x; j < mine; j += kRouteThreads) {
    double v = slices[j * cuts];
    for (int c = 1; c < cuts; ++c) v += slices[j * cuts + c];
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to + (uint32_t)(rank + j * ranks) * 8u),
                 "d"(v)
                 : "memory");
  }
  cluster_sync();
  if (rank == 0 && warp == 0) token_choice(a, t, logits);
}

// The lists of every CTA from the choices: a counting sort by expert.  `scratch` (the
// ring, not in use yet): [chunks of 32 pairs][E] counts, then each pair's expert and its
// place among its chunk's.
__device__ void build_lists(const MoeKArgs& a, const Lists& L, uint16_t* scratch, Line* line,
                            Walk* walk) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = a.T * a.topk, chunks = (P + 31) / 32;
  uint16_t* hist = scratch;
  uint16_t* expert = hist + (chunks * a.E + 1) / 2 * 2;
  uint16_t* place = expert + chunks * 32;
  for (int i = tid; i < (chunks * a.E + 1) / 2; i += kThreads)
    reinterpret_cast<uint32_t*>(hist)[i] = 0u;
  __syncthreads();
#pragma unroll 4
  for (int c = warp; c < chunks; c += kWarps) {
    const int p = c * 32 + lane;
    const int e = p < P ? __ldcg(a.idx + p) : -1;
    const unsigned m = __match_any_sync(0xffffffffu, e);
    if (p < P) {
      const int before = __popc(m & ((1u << lane) - 1u));
      expert[p] = (uint16_t)e;
      place[p] = (uint16_t)before;
      if (before == 0) hist[c * a.E + e] = (uint16_t)__popc(m);
    }
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kThreads) {
    int n = 0;
    for (int c = 0; c < chunks; ++c) {
      const int q = hist[c * a.E + e];
      hist[c * a.E + e] = (uint16_t)n;
      n += q;
    }
    L.count[e] = n;
  }
  __syncthreads();
  if (warp == 0) {   // running sums of rows and of blocks over the experts
    int rows = 0, blocks = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane, n = e < a.E ? L.count[e] : 0, nb = (n + a.NB - 1) / a.NB;
      int r = n, b = nb;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int r2 = __shfl_up_sync(0xffffffffu, r, o), b2 = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
          r += r2;
          b += b2;
        }
      }
      if (e < a.E) {
        L.first[e] = rows + r - n;
        L.block[e] = (uint16_t)(blocks + b - nb);
        for (int i = 0; i < nb; ++i)
          L.entry[blocks + b - nb + i] = {(uint16_t)e, (uint16_t)(rows + r - n + i * a.NB),
                                          (uint16_t)min(a.NB, n - i * a.NB), 0};
      }
      rows += __shfl_sync(0xffffffffu, r, 31);
      blocks += __shfl_sync(0xffffffffu, b, 31);
    }
    if (lane == 0) *L.n_entries = blocks;
  }
  __syncthreads();
  if (warp >= 6) {   // the phases' lines and this CTA's ranges
    // Partial tiles cost the first phase a round of counting and of h, 4 us, and their sums
    // more with more rows (53 tokens, 2 experts of 2208 x 1864: 8 parts at most 36 us, 4 33
    // us); the second sums them where it has to wait anyway.
    const Line l = warp == 6 ? make_line(*L.n_entries, a.F, a.D, 128, 4.0f, a.NB <= 32 ? 3 : 2)
                             : make_line(*L.n_entries, a.D, a.F, 256, 1.0f, 4);
    const Walk w(l);
    if (lane == 0) {
      line[warp - 6] = l;
      walk[warp - 6] = w;
    }
  }
  for (int p = tid; p < P; p += kThreads) {
    const int e = expert[p], at = hist[(p >> 5) * a.E + e] + place[p], r = L.first[e] + at;
    L.token[r] = (uint16_t)(p / a.topk);
    L.ent[r] = (uint16_t)(L.block[e] + at / a.NB);
    L.row[p] = (uint16_t)r;
  }
  fence_proxy_async_smem();   // TMA writes over the scratch
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
  constexpr int U = 2;   // items whose loads are in flight together
  const unsigned nseg = c1 - c0 + 1, total = en.n * 32u, step = nseg * 128;
  for (unsigned i0 = (blockIdx.x - c0) * 128 + et; i0 < total; i0 += U * step) {
    float4 g[U], u[U];
    int64_t at[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const unsigned i = min(i0 + q * step, total - 1);
      at[q] = (int64_t)(i >> 5) * 256 + (i & 31) * 4;
      const float* p = part_of(a, 0, c0, 1) + at[q];
      g[q] = ld4(p);
      u[q] = ld4(p + 128);
    }
#pragma unroll 4
    for (unsigned c = c0 + 1; c <= c1; ++c) {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const float* p = part_of(a, 0, c, 0) + at[q];
        add4(g[q], ld4(p));
        add4(u[q], ld4(p + 128));
      }
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const unsigned i = i0 + q * step, col = tile * 128 + (i & 31) * 4;
      if (i < total && col < (unsigned)a.F)
        *reinterpret_cast<uint2*>(a.h + (int64_t)(en.r0 + (i >> 5)) * a.F + col) =
            make_uint2(pack2(glu(g[q].x, u[q].x), glu(g[q].y, u[q].y)),
                       pack2(glu(g[q].z, u[q].z), glu(g[q].w, u[q].w)));
    }
  }
}

// out of every token: its experts' products weighted in the order of the choices, by
// groups of 4 columns.
struct OutGroup {
  unsigned t, d;   // token, first column
  uint2 res;
  float4 sum;
  __device__ __forceinline__ void start(const MoeKArgs& a, unsigned i) {
    const unsigned d4 = (unsigned)a.D / 4;
    t = i / d4;
    d = (i - t * d4) * 4;
    res = make_uint2(0u, 0u);
    if (a.residual) res = reinterpret_cast<const uint2*>(a.residual)[i];
    sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  template <typename W>
  __device__ __forceinline__ void add(const W& term, const float4& v) {
    sum.x = fmaf(term.w, v.x, sum.x);
    sum.y = fmaf(term.w, v.y, sum.y);
    sum.z = fmaf(term.w, v.z, sum.z);
    sum.w = fmaf(term.w, v.w, sum.w);
  }
  __device__ __forceinline__ void store(const MoeKArgs& a, unsigned i) const {
    reinterpret_cast<uint2*>(a.out)[i] =
        make_uint2(pack2(sum.x + __uint_as_float(res.x << 16),
                         sum.y + __uint_as_float(res.x & 0xffff0000u)),
                   pack2(sum.z + __uint_as_float(res.y << 16),
                         sum.w + __uint_as_float(res.y & 0xffff0000u)));
  }
};

// The product of a group with its token's c-th expert: in y, or in partial tiles.
struct Term {
  const float* p;
  const float* next;
  unsigned more;
  float w;
  __device__ __forceinline__ void find(const MoeKArgs& a, const Lists& L, const Line& l,
                                       const OutGroup& o, int c) {
    const unsigned pair = o.t * a.topk + c;
    const int r = L.row[pair], ent = L.ent[r];
    w = a.wgt[pair];
    unsigned c0, c1;
    l.ctas_of(ent * l.tiles + (o.d >> 8), c0, c1);
    const int64_t at = (int64_t)(r - L.entry[ent].r0) * 256 + (o.d & 255);
    p = c0 == c1 ? a.y + r * (int64_t)l.tiles * 256 + o.d : part_of(a, 1, c0, 1) + at;
    next = part_of(a, 1, c0 + 1, 0) + at;
    more = c1 - c0;
  }
  __device__ __forceinline__ void none() {
    p = next = nullptr;
    more = 0u;
    w = 0.0f;
  }
};

// The products of N terms, each the sum of its partial tiles in order, with the loads of all
// of them in flight together (one after another they took 9 us of 200 tokens' 38 us).
template <int N>
__device__ __forceinline__ void products(const MoeKArgs& a, const Term (&t)[N], float4 (&v)[N]) {
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int64_t step = (int64_t)a.NB * 512;   // from a CTA's partial tile to the next one's
  unsigned most = 0;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = t[n].p ? ld4(t[n].p) : zero;
    most = max(most, t[n].more);
  }
  for (unsigned k = 0; k < most; k += 4) {
    float4 q[N][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int n = 0; n < N; ++n)
        q[n][j] = k + j < t[n].more ? ld4(t[n].next + (k + j) * step) : zero;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int n = 0; n < N; ++n) add4(v[n], q[n][j]);
  }
}

// Two groups a thread and two of their experts at a time.
__device__ __forceinline__ void form_out(const MoeKArgs& a, const Lists& L, const Line& l) {
  constexpr int U = 2;
  const unsigned total = (unsigned)a.T * (a.D / 4), step = gridDim.x * kThreads;
  for (unsigned i0 = blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += U * step) {
    OutGroup o[U];
#pragma unroll
    for (int u = 0; u < U; ++u) o[u].start(a, min(i0 + u * step, total - 1));
    for (int c = 0; c < a.topk; c += 2) {
      Term term[2 * U];
      float4 v[2 * U];
#pragma unroll
      for (int u = 0; u < 2 * U; ++u) {
        if (c + (u & 1) < a.topk && i0 + (u >> 1) * step < total)
          term[u].find(a, L, l, o[u >> 1], c + (u & 1));
        else
          term[u].none();
      }
      products(a, term, v);
#pragma unroll
      for (int u = 0; u < 2 * U; ++u) o[u >> 1].add(term[u], v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * step < total) o[u].store(a, i0 + u * step);
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
  __shared__ int out_flag;
  __shared__ int4 gather_rows[2][32];   // token rows of the block, 4 a gather
  __shared__ Line line[2];   // of the phases
  __shared__ Walk walk[2];
  const Lists L(smem + S * stage_bytes, a.T * a.topk, a.E, a.NB);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t tmem_cols = 64;   // two accumulators of two row groups
  while (tmem_cols < 4u * a.NB) tmem_cols *= 2;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 3);    // the weights' and two of the tokens' producers
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
  build_lists(a, L, reinterpret_cast<uint16_t*>(smem), line, walk);
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (elect_one()) {
      const uint64_t pol = l2_evict_first_policy();   // weights pass through once
      const uint32_t base = smem_u32(smem);
      Place at;
      bool ok = true;
      for (int ph = 0; ok && ph < 2; ++ph) {
        for (Walk w = walk[ph]; ok && w.more(); w.next()) {
          const int e = L.entry[w.ent].e, row = (int)w.tile * (ph == 0 ? 128 : 256);
          int k = (int)w.k * kK;
          for (unsigned n = w.steps(); n > 0; --n, k += kK, at.next(S)) {
            // (the first round's wait for "empty" returns at once)
            if (!mbar_wait(smem_u32(&empty[at.s]), at.parity ^ 1u, a.err, 92)) {
              ok = false;
              break;
            }
            const uint32_t fb = smem_u32(&full[at.s]), dst = base + at.s * stage_bytes;
            mbar_arrive_expect_tx(fb, kWBytes);
            if (ph == 0) {
              tma_load_3d(dst, &tm_wg, fb, k, row, e, pol);
              tma_load_3d(dst + kSlabBytes, &tm_wu, fb, k, row, e, pol);
            } else {
              tma_load_3d(dst, &tm_wd, fb, k, row, e, pol);
              tma_load_3d(dst + kSlabBytes, &tm_wd, fb, k, row + 128, e, pol);
            }
          }
        }
      }
    }
  } else if (warp >= 6) {
    const int half = warp - 6;
    const uint32_t base = smem_u32(smem) + kWBytes;
    Place at;
    bool ok = true;
    for (int ph = 0; ok && ph < 2; ++ph) {
      unsigned have = ~0u;   // the block whose h is known to be there, or whose rows are held
      for (Walk w = walk[ph]; ok && w.more(); w.next()) {
        const Entry en = L.entry[w.ent];
        // this warp's blocks of 16 rows
        const int n16 = (en.n + 15) / 16, b0 = half ? (n16 + 1) / 2 : 0;
        const int b1 = half ? n16 : (n16 + 1) / 2;
        if (w.ent != have) {
          have = w.ent;
          if (ph == 0) {
            // rows behind the last repeat it (their columns of the accumulator are not read)
            __syncwarp();
            const uint16_t* tok = L.token + en.r0;
            const int r = lane * 4, last = en.n - 1;
            gather_rows[half][lane] = make_int4(tok[min(r, last)], tok[min(r + 1, last)],
                                                tok[min(r + 2, last)], tok[min(r + 3, last)]);
            __syncwarp();
          } else {
            ok = warp_wait(&a.sync->ready[w.ent], line[0].tiles * line[0].ksteps, a.err, 93);
            if (!ok) break;
            fence_proxy_async_global();
          }
        }
        int fail = 0;
        if (elect_one()) {
          int k = (int)w.k * kK;
          Place p = at;
          for (unsigned n = w.steps(); n > 0; --n, k += kK, p.next(S)) {
            if (!mbar_wait(smem_u32(&empty[p.s]), p.parity ^ 1u, a.err, 94)) {
              fail = 1;
              break;
            }
            const uint32_t fb = smem_u32(&full[p.s]), dst = base + p.s * stage_bytes;
            mbar_arrive_expect_tx(fb, (uint32_t)((b1 - b0) * 16 * 128));
            if (ph == 0) {
              for (int q = b0 * 4; q < b1 * 4; q += 2) {   // 4 rows by index at a time
                const int4 t = gather_rows[half][q], u = gather_rows[half][q + 1];
                tma_gather4(dst + q * 512, &tm_x, fb, k, t.x, t.y, t.z, t.w);
                tma_gather4(dst + q * 512 + 512, &tm_x, fb, k, u.x, u.y, u.z, u.w);
              }
            } else {
              for (int q = b0; q < b1; ++q) tma_load_2d(dst + q * 2048, &tm_h, fb, k, en.r0 + q * 16);
            }
          }
        }
        at.skip(w.steps(), S);   // every lane keeps the place
        ok = !__any_sync(0xffffffffu, fail);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint64_t ring = sw128_kmajor_desc(smem_u32(smem));
      Place at, acc;
      bool ok = true;
      for (int ph = 0; ok && ph < 2; ++ph) {
        for (Walk w = walk[ph]; ok && w.more(); w.next(), acc.next(2)) {
          const int n16 = (L.entry[w.ent].n + 15) / 16;
          const uint32_t idesc = idesc_bf16_f32(128, n16 * 16);
          if (!mbar_wait(smem_u32(&acc_empty[acc.s]), acc.parity ^ 1u, a.err, 95)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + acc.s * (uint32_t)(2 * a.NB);
          uint32_t add = 0u;
          for (unsigned n = w.steps(); n > 0; --n, at.next(S)) {
            if (!mbar_wait(smem_u32(&full[at.s]), at.parity, a.err, 96)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t wd = ring + at.s * (unsigned)(stage_bytes / 16);
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int kk = 0; kk < kK / 16; ++kk)
                umma_f16(d + (uint32_t)(g * a.NB), wd + (g * kSlabBytes + kk * 32) / 16,
                         wd + (kWBytes + kk * 32) / 16, idesc, kk > 0 ? 1u : add);
            add = 1u;
            umma_commit(smem_u32(&empty[at.s]));
          }
          if (ok) umma_commit(smem_u32(&acc_full[acc.s]));
        }
      }
    }
  } else {
    const int lg = warp & 3, et = lg * 32 + lane;   // TMEM lane = weight row of a group
    Place acc;
    bool ok = true;
    for (int ph = 0; ok && ph < 2; ++ph) {
      const Line& l = line[ph];
      for (Walk w = walk[ph]; w.more(); w.next(), acc.next(2)) {
        const unsigned ent = w.ent, tile = w.tile, b = acc.s;
        const bool whole = w.whole();
        const Entry en = L.entry[ent];
        if (!mbar_wait(smem_u32(&acc_full[b]), acc.parity, a.err, 97)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem + ((uint32_t)(lg * 32) << 16) + b * (uint32_t)(2 * a.NB);
        float* dst = part_of(a, ph, blockIdx.x, w.k == 0 ? 1 : 0) + et;
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
              // (all 16 first, so that they overlap; rows behind the last are not stored)
              __nv_bfloat16 hv[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                hv[i] = __float2bfloat16_rn(glu(__uint_as_float(g[i]), __uint_as_float(q[i])));
              const int n = en.n - c;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (i < n) *hp = hv[i];
                hp += a.F;
              }
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
      }
      if (ph == 0) {
        // What others wait for is counted once, behind one fence: a fence after each unit
        // held the drain up for 2 us of every 4 with units of 3 steps.
        fence_proxy_async_global();   // h is read by TMA
        ok = epi_all(ok);
        // The cut units this CTA took part in are its first and its last.
        unsigned cut_u[2], cut_steps[2], block = ~0u, done = 0;
        int cuts = 0;
        for (Walk w = walk[ph]; ok && w.more(); w.next()) {
          const unsigned u = w.ent * w.tiles + w.tile;
          if (w.whole()) {   // counted for all units of a block at once
            if (w.ent != block && done) {
              if (et == 0) add_release(&a.sync->ready[block], done);
              done = 0;
            }
            block = w.ent;
            done += w.ksteps;
          } else {
            unsigned c0, c1;
            l.ctas_of(u, c0, c1);
            cut_u[cuts] = u;
            cut_steps[cuts++] = w.steps();
            if (et == 0) add_release(&a.sync->unit[c0], w.steps());
          }
        }
        if (done && et == 0) add_release(&a.sync->ready[block], done);
        // Its share of them.
        for (int i = 0; ok && i < cuts; ++i) {
          unsigned c0, c1;
          l.ctas_of(cut_u[i], c0, c1);
          ok = warp_wait(&a.sync->unit[c0], l.ksteps, a.err, 98);
          const unsigned ent = cut_u[i] / l.tiles;
          if (ok) join_h(a, L.entry[ent], cut_u[i] - ent * l.tiles, c0, c1, et);
        }
        if (cuts) {
          fence_proxy_async_global();
          ok = epi_all(ok);
          for (int i = 0; ok && et == 0 && i < cuts; ++i)
            add_release(&a.sync->ready[cut_u[i] / l.tiles], cut_steps[i]);
        }
      }
    }
    epi_add(&a.sync->done, 1, et);
  }
  // The last sum.  Where a thread has one group of columns at most, what it needs for the
  // first two experts is looked up before the wait.
  const unsigned groups = (unsigned)a.T * (a.D / 4), mine = blockIdx.x * kThreads + tid;
  const bool few = groups <= gridDim.x * kThreads, has = few && mine < groups;
  OutGroup o;
  Term term[2];
  if (has) {
    o.start(a, mine);
    term[0].find(a, L, line[1], o, 0);
    if (a.topk > 1)
      term[1].find(a, L, line[1], o, 1);
    else
      term[1].none();
  }
  if (tid == 64)
    out_flag = wait_count(&a.sync->done, gridDim.x, a.err, 99) ? 1 : 0;
  tc_fence_before();
  __syncthreads();
  if (out_flag) {
    if (has) {
      for (int c = 0; c < a.topk; c += 2) {
        if (c > 0) {
          term[0].find(a, L, line[1], o, c);
          if (c + 1 < a.topk)
            term[1].find(a, L, line[1], o, c + 1);
          else
            term[1].none();
        }
        float4 v[2];
        products(a, term, v);
        o.add(term[0], v[0]);
        if (c + 1 < a.topk) o.add(term[1], v[1]);
      }
      o.store(a, mine);
    } else if (!few) {
      form_out(a, L, line[1]);
    }
  }
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
  const int nb = (int)ceil_div(want, 16) * 16;
  return nb < 16 ? 16 : nb < kMaxBlock ? nb : kMaxBlock;
}

constexpr size_t kSmemMost = 227 * 1024;
constexpr size_t kStaticMost = 1536;  // barriers, flags and gather rows
int ring_stages(int nb, size_t lists) {
  const size_t n = (kSmemMost - kStaticMost - 1024 - lists) / (kWBytes + nb * 128);
  return n > kMaxStages ? kMaxStages : (int)n;
}

size_t ring_smem(int nb, size_t lists) {
  return 1024 + ring_stages(nb, lists) * (size_t)(kWBytes + nb * 128) + lists;
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
  const size_t lists = Lists::bytes(a.T * a.topk, a.E, a.NB);
  a.stages = ring_stages(a.NB, lists);
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
  // CTAs a token's experts are shared by: up to 8, while the grid stays below two waves
  int ranks = 8;
  while (ranks > 1 && (ranks > m.E || m.T * ranks > 2 * ctas)) ranks /= 2;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.stream = p.stream;
  cfg.gridDim = dim3((unsigned)ranks, (unsigned)m.T);
  cfg.blockDim = dim3(kRouteThreads);
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_moe_route, a);
  if (e != cudaSuccess) return e;
  launched(p, "k_moe_route");
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = ring_smem(a.NB, lists);
  e = cudaLaunchKernelEx(&cfg, k_moe, wg, wu, wd, tx, th, a);
  if (e == cudaSuccess) launched(p, "k_moe");
  return e;
}

}  // namespace jmix
