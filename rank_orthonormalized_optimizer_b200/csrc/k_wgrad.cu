// The gradient of a 2-D weight from activations kept in 8 bits:
//
//   G = A^T D   (m x n)      or, output-major,   G^T = D^T A   (n x m)
//
// A [tokens, m] are e4m3 bytes with a power-of-two scale per 32 features (rows.cuh), D
// [tokens, n] bf16 gradients of the layer's output, G fp32: what the optimizer step reads.
//
// A's values are exact in bf16 and so are the products in fp32; the only roundings are the
// fp32 additions.  There are two kernels.  Where G has few columns, k_wgrad reads the 8-bit rows
// and converts each tile on its way; where it has many, each feature's tile would be converted
// once for every 256 columns, and the conversion's shared-memory traffic and power take a sixth of
// the tensor cores' rate (m = 4096, n = 11008, 16384 tokens: 1247 us against 1026, 1440 TFLOP/s, in
// short runs; 1458 against 1237 repeated, under the power cap): there A is first brought to bf16
// rows in the workspace (dion_act_load) and k_wgrad_rows, whose tensor pipe is 90 % busy,
// multiplies those.
//
// The contraction over the tokens runs on the tensor cores: a persistent pair
// of CTAs (a cluster, tcgen05 cta_group::2) owns 256 x BN tiles of G, each CTA 128 of the
// features and half of the columns, and walks the tokens 64 at a time.  In each CTA
//   warp 0        TMA producer of the 8-bit tile (64 tokens x 128 features)
//   warp 1        MMA issuer (one thread, in the pair's first CTA)
//   warp 2        TMEM allocator; TMA producer of the CTA's half of the D tile
//   warp 3        the tile's scale bytes (cp.async)
//   warps 4..15   converters: e4m3 and scale -> bf16, written as the 128-byte-swizzled
//                 MN-major operand that tcgen05.mma reads; three groups of four take turns,
//                 so that one group's latencies pass behind the others' work
//   warps 16..23  epilogue
// The tensor cores' accumulation rounds toward zero, which adds up over thousands of MMAs,
// so the tokens are cut into chunks of kChunk blocks, each accumulated from zero in TMEM
// (two accumulators in turn), and the epilogue warps add the chunks in fp32 registers: over
// 16384 like-signed products 3e-7 off (an fp32 product on CUDA cores 6e-7; chunks of 8 blocks 1.3e-7
// and 2.5 % slower, of 4 8e-8 and 7 %: k_wgrad at m = 4096, n = 11008 in one run).
// The tiles that do not fill a last round over all pairs (all of them, in a small matrix) are
// also split over the tokens, so that every pair has a share; their partial sums go to the
// workspace and a second kernel adds them in order.  Every wait is bounded; after a give-up the
// CTA lets its loads and MMAs end, marks DION_MAT_TIMEOUT and leaves what it has not finished of G
// as it was.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "operator.h"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace dion {
namespace {

using namespace tc;

constexpr int BM = 128;      // features of A per CTA = TMEM lanes
constexpr int PM = 2 * BM;   // features of a pair's tile
constexpr int BK = 64;       // tokens per stage
constexpr int kChunk = 16;   // stages per accumulation chunk
constexpr int NT = 32 * (4 + 12 + 8);
constexpr int SQ = 6;        // stages of the 8-bit tiles
constexpr int SB = 6;        // stages of the D tiles
constexpr int SA = 4;        // stages of the converted operand
constexpr int kGroups = 3, kGroupWarps = 4;                // converters
// A converter group waits for a stage's barrier by its parity alone, so the stage that used the
// slot before must be known to be full by then: it is the group's own when SQ is a multiple of
// kGroups.  (Of the converted ring, a group's last wait says that all MMAs up to SA stages
// before its last stage are done, which covers the slot's previous use when SA >= kGroups;
// the MMAs it knows done had their D tiles, which covers D's slots when SB >= SA.)
static_assert(SQ % kGroups == 0 && SA >= kGroups && SB >= SA, "a slot's previous phase must be over");
constexpr int kItems = BK * BM / 16 / (32 * kGroupWarps);  // 16-feature groups per thread
constexpr int Q_BYTES = BK * BM;
constexpr int A_BYTES = BK * BM * 2;

struct WgradP {
  const uint8_t* scale;
  float* out;        // G
  float* parts;      // [tail tile][split][PM][BN]: partial sums of the split tiles
  int32_t* gave_up;  // [CTA]: whether a wait of it ran out in this call (null without a join)
  int32_t* status;
  int64_t tokens, ld_scale, ldg, m, n;
  int tiles_m, whole, tail;               // tiles taken whole, and split over the tokens
  int splits, blocks_per_split, blocks;   // blocks: of 64 tokens
  int transposed, accumulate, vec;
  int ctas;          // of the kernel
  int scale4;        // the scale bytes of a tile's token are an aligned word
  int64_t max_spins;
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                            int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// A lane's 8 floats of its row, a whole 32-byte sector: the lanes of a warp write 32 rows, and
// two 16-byte halves would reach L2 as two partial sectors.
__device__ __forceinline__ void store_sector(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
template <int R> __device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R> __device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// ---- the pair: barriers of the first CTA, MMAs and TMEM of both
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the same barrier in the pair's first CTA
__device__ __forceinline__ uint32_t first_cta(uint64_t* bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
  return r;
}
// What an arrival hands over lies in the arriver's own shared memory (ordered before it by the
// proxy fence) or in TMEM (by the tcgen05 fences), so the CTA-scope default is enough; with
// cluster-scope release and acquire each arrival waited about 1600 cycles for every earlier
// memory operation of its thread, and the kernel ran at 690 TFLOP/s.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Arrive on `bar` of both CTAs once the MMAs issued so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// The last `stages` of the `issued` loads into a ring have landed.
__device__ __forceinline__ void wait_landed(uint64_t* full, int stages, int issued) {
  for (int j = max(0, issued - stages); j < issued; ++j) wait_drain(full + j % stages, (uint32_t)(j / stages) & 1);
}
// After a give-up, once every role of this CTA has stopped: the same for the 8-bit ring, whose
// barriers also wait for the scale warp.  Either of the two may have gone further than the other;
// the arrivals that are missing are made here, where nobody reads the tiles any more.
__device__ __forceinline__ void land_scaled(uint64_t* full, int stages, int tiles, int scales) {
  const int most = max(tiles, scales);
  for (int j = max(0, most - stages); j < most; ++j) {
    if (j >= tiles) mbar_arrive(full + j % stages);
    for (int k = 0; k < 32 && j >= scales; ++k) mbar_arrive(full + j % stages);
  }
  wait_landed(full, stages, most);
}

// Four e4m3 bytes to bf16 times `f`: bytes 0 and 2 to `even`, 1 and 3 to `odd`.  A byte's 7
// magnitude bits, moved to bf16's exponent and fraction, read as its value times 2^-120
// (subnormals too: both formats count them in steps of their smallest normal).  f carries the
// 2^120; all products are exact, being by powers of two.  Taking every other byte needs no
// byte permutation; the features' order in the tile is then 0 2 1 3 of each four, which the
// epilogue undoes.
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void e4m3x4_bf16(uint32_t w, uint32_t f, uint32_t& even, uint32_t& odd) {
  constexpr uint32_t M = 0x07f007f0u;   // the magnitude's place
  const uint32_t s = w & 0x80808080u;   // signs; the other pair's fall inside M, and out
  even = bf16x2_mul(((w << 4) & M) | ((s << 8) & ~M), f);
  odd = bf16x2_mul(((w >> 4) & M) | (s & ~M), f);
}

// A unit of work: one tile over one range of token blocks; part: where its partial sums go
// (-1: the whole sum, straight to G).
struct Unit {
  int m0, n0, part, kb0, kb1;
};
template <int BN>
__device__ __forceinline__ Unit unit_of(const WgradP& p, int u) {
  Unit t;
  int tile = u;
  t.part = -1;
  t.kb0 = 0;
  t.kb1 = p.blocks;
  if (u >= p.whole) {
    t.part = u - p.whole;
    tile = p.whole + t.part / p.splits;
    t.kb0 = t.part % p.splits * p.blocks_per_split;
    t.kb1 = min(p.blocks, t.kb0 + p.blocks_per_split);
  }
  t.m0 = tile % p.tiles_m * PM;
  t.n0 = tile / p.tiles_m * BN;
  return t;
}

// The epilogue of one warp: 32 features and half of the tile's columns; `place` is the feature of
// its TMEM lane.  Chunks are added in registers, the sum is written once.
template <int BN>
__device__ __forceinline__ void epilogue(const WgradP& p, float* staging, uint32_t tmem, uint64_t* tfull,
                                         uint64_t* tempty, volatile int* abort, int ew, int lane, int place,
                                         int rank, int pair, int pairs) {
  constexpr int HB = BN / 2;
  const int units = p.whole + p.tail * p.splits;
  const int row0 = (ew & 3) * 32;
  const int col0 = (ew >> 2) * HB;
  int acc = 0;
  uint32_t pacc = 0;
  bool ok = true;
  for (int u = pair; u < units && ok; u += pairs) {
    const Unit t = unit_of<BN>(p, u);
    float run[HB];
#pragma unroll
    for (int i = 0; i < HB; ++i) run[i] = 0.f;
    for (int c0 = t.kb0; c0 < t.kb1; c0 += kChunk) {
      const bool w = wait_bounded(tfull + acc, pacc, p.max_spins, abort);
      if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
      tc_fence_after();
      const uint32_t base = tmem + ((uint32_t)row0 << 16) + acc * BN + col0;
#pragma unroll
      for (int c = 0; c < HB; c += 8) {
        float v[8];
        tmem_ld8(base + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) run[c + i] += v[i];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(first_cta(tempty + acc));
      acc ^= 1;
      if (acc == 0) pacc ^= 1;
    }
    if (!ok) break;
    const int64_t row = t.m0 + rank * BM + row0 + place;
    const int64_t n0 = t.n0 + col0;
    if (t.part >= 0) {
      float* g = p.parts + ((int64_t)t.part * PM + rank * BM + row0 + place) * BN + col0;
#pragma unroll
      for (int i = 0; i < HB; i += 8) store_sector(g + i, run + i);
    } else if (p.transposed) {
      // 32 lanes write 32 neighbouring features of one column
#pragma unroll
      for (int i = 0; i < HB; ++i)
        if (row < p.m && n0 + i < p.n) {
          float* g = p.out + (n0 + i) * p.ldg + row;
          *g = run[i] + (p.accumulate ? *g : 0.f);
        }
    } else {
      float* g = p.out + min(row, p.m - 1) * p.ldg + n0;
#pragma unroll
      for (int i = 0; i < HB; i += 8) {
        if (!p.vec) {
          // rows that do not start on a sector: through shared memory, so that eight lanes write
          // a row's eight columns instead of 32 lanes 32 rows
          float* buf = staging + ew * 32 * 9;
#pragma unroll
          for (int j = 0; j < 8; ++j) buf[place * 9 + j] = run[i + j];
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int64_t r = t.m0 + rank * BM + row0 + 4 * k + (lane >> 3), col = n0 + i + (lane & 7);
            if (r < p.m && col < p.n) {
              float* to = p.out + r * p.ldg + col;
              const float v = buf[(4 * k + (lane >> 3)) * 9 + (lane & 7)];
              *to = v + (p.accumulate ? *to : 0.f);
            }
          }
          __syncwarp();
        } else if (row >= p.m) {
          // a lane past the last feature writes nothing
        } else if (n0 + i + 7 < p.n) {
          if (p.accumulate) {
            const float4 a = *reinterpret_cast<const float4*>(g + i), b = *reinterpret_cast<const float4*>(g + i + 4);
            run[i] += a.x; run[i + 1] += a.y; run[i + 2] += a.z; run[i + 3] += a.w;
            run[i + 4] += b.x; run[i + 5] += b.y; run[i + 6] += b.z; run[i + 7] += b.w;
          }
          store_sector(g + i, run + i);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (n0 + i + j < p.n) g[i + j] = run[i + j] + (p.accumulate ? g[i + j] : 0.f);
        }
      }
    }
    __syncwarp();  // the next unit's TMEM loads are warp-wide
  }
  if ((!ok || *abort) && lane == 0 && p.status) atomicOr(p.status, F_TIMEOUT);
}

// Shared memory of a CTA: the rings, the barriers, and the epilogue's staging.
template <int BN> struct Smem {
  static constexpr int rings = SA * A_BYTES + SB * BK * BN + SQ * (Q_BYTES + 2 * BK * 4);
  static constexpr int epilogue = rings + 512;  // the barriers in between
  static constexpr int bytes = 1024 + epilogue + 8 * 32 * 9 * 4;
  static_assert((2 * SQ + 2 * SB + 2 * SA + 5) * 8 + 24 <= 512, "the barriers");
  static_assert(bytes <= 227 * 1024, "shared memory");
};

template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NT, 1)
    k_wgrad(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmD,
            const WgradP p) {
  constexpr int HB = BN / 2;               // columns of D that a CTA loads
  constexpr int B_BYTES = BK * HB * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);     // the same offset in both CTAs
  uint8_t* sA = smem;
  uint8_t* sB = sA + SA * A_BYTES;
  uint8_t* sQ = sB + SB * B_BYTES;
  uint32_t* sS = reinterpret_cast<uint32_t*>(sQ + SQ * Q_BYTES);  // [stage][2][token]: scale bytes
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sS + SQ * 2 * BK);   // the 8-bit tile and its scales
  uint64_t* q_empty = q_full + SQ;
  uint64_t* b_full = q_empty + SQ;
  uint64_t* b_empty = b_full + SB;
  uint64_t* a_full = b_empty + SB;         // used in the first CTA
  uint64_t* a_empty = a_full + SA;
  uint64_t* tfull = a_empty + SA;
  uint64_t* tempty = tfull + 2;            // used in the first CTA
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = abort + 1;        // stages of the 8-bit ring: tiles, scales
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int units = p.whole + p.tail * p.splits;
  constexpr uint32_t kCols = 2 * BN;  // TMEM columns: two accumulators

  if (threadIdx.x == 0) {
    for (int s = 0; s < SQ; ++s) {
      mbar_init(q_full + s, 1 + 32);  // the TMA producer's arrival and the scale warp's lanes
      mbar_init(q_empty + s, kGroupWarps);
    }
    for (int s = 0; s < SB; ++s) {
      mbar_init(b_full + s, 1);
      mbar_init(b_empty + s, 1);
    }
    for (int s = 0; s < SA; ++s) {
      mbar_init(a_full + s, 2 * kGroupWarps);  // of both CTAs
      mbar_init(a_empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tempty + a, 2 * 8);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc_pair(tmem_slot, kCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  grid_trigger();  // a grid of one round: the join's CTAs come as these end
  // (by a thread without a role, so that nothing waits for the store)
  if (threadIdx.x == 33 && p.gave_up) p.gave_up[blockIdx.x] = 0;
  if (warp < 4) {
    reg_dec<40>();
    if ((warp == 0 || warp == 2) && lane == 0) {
      // ---------------- TMA producers, one for each operand: the 8-bit tiles must not wait for
      // the MMAs that hold D's slots, since they have to be converted first
      const bool q = warp == 0;
      const CUtensorMap* map = q ? &tmQ : &tmD;
      uint64_t *fullb = q ? q_full : b_full, *emptyb = q ? q_empty : b_empty;
      const int stages = q ? SQ : SB;
      prefetch_map(map);
      int stage = 0, count = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        const Unit t = unit_of<BN>(p, u);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++count) {
          if (!wait_bounded(emptyb + stage, phase ^ 1, p.max_spins, abort)) { ok = false; break; }
          mbar_expect_tx(fullb + stage, q ? Q_BYTES : B_BYTES);
          if (q) {
            tma_load_2d(sQ + stage * Q_BYTES, map, fullb + stage, t.m0 + rank * BM, kb * BK);
          } else {
#pragma unroll
            for (int j = 0; j < HB / 64; ++j)
              tma_load_2d(sB + stage * B_BYTES + j * 8192, map, fullb + stage,
                          t.n0 + rank * HB + 64 * j, kb * BK);
          }
          if (++stage == stages) { stage = 0; phase ^= 1; }
        }
      }
      // every load issued lands before the CTA goes away, whichever role gives up
      if (q) issued[0] = count;
      else wait_landed(fullb, stages, count);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---------------- MMA issuer of the pair: a stage is ready once the converters of both
      // CTAs, who waited for its D tile too, have arrived
      constexpr uint32_t idesc = idesc_bf16(PM, BN, true, true);
      int sb = 0, sa = 0, acc = 0;
      uint32_t pa = 0, pacc = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        const Unit t = unit_of<BN>(p, u);
        for (int c0 = t.kb0; c0 < t.kb1 && ok; c0 += kChunk) {
          if (!wait_bounded(tempty + acc, pacc ^ 1, p.max_spins, abort)) { ok = false; break; }
          tc_fence_after();
          const int c1 = min(t.kb1, c0 + kChunk);
          for (int kb = c0; kb < c1; ++kb) {
            if (!wait_bounded(a_full + sa, pa, p.max_spins, abort)) { ok = false; break; }
            tc_fence_after();
            const uint32_t ab = smem_u32(sA + sa * A_BYTES), bb = smem_u32(sB + sb * B_BYTES);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              mma_pair(tmem + acc * BN, sw128_desc(ab + k * 2048, 8192, 1024),
                       sw128_desc(bb + k * 2048, 8192, 1024), idesc, ((kb - c0) | k) != 0);
            commit_pair(b_empty + sb);
            commit_pair(a_empty + sa);
            if (++sb == SB) sb = 0;
            if (++sa == SA) { sa = 0; pa ^= 1; }
          }
          if (!ok) break;
          commit_pair(tfull + acc);
          acc ^= 1;
          if (acc == 0) pacc ^= 1;
        }
      }
      commit_pair(drain);
      wait_drain(drain, 0);
    } else if (warp == 3) {
      // ---------------- scale bytes: the word of a token's four, or the two words that they
      // lie in, two tokens a lane
      const uintptr_t begin = reinterpret_cast<uintptr_t>(p.scale), end = begin + p.tokens * p.ld_scale;
      int stage = 0, count = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        const Unit t = unit_of<BN>(p, u);
        const int64_t c = (t.m0 + rank * BM) / DION_ACT_BLOCK;
        const int valid = (int)min((int64_t)4, max((int64_t)0, p.ld_scale - c));  // bytes of a token
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          ok = __all_sync(0xffffffffu, wait_bounded(q_empty + stage, phase ^ 1, p.max_spins, abort));
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int64_t tok = (int64_t)kb * BK + lane + 32 * i;
            const uintptr_t at = begin + (tok < p.tokens && valid > 0 ? tok * p.ld_scale + c : 0);
            const int bytes = tok < p.tokens ? valid : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == 1 && p.scale4) break;
              const uintptr_t word = (at & ~(uintptr_t)3) + 4 * h;
              const uint32_t to = smem_u32(sS + (stage * 2 + h) * BK + lane + 32 * i);
              if (bytes == 0 || word >= at + bytes) {
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(0u) : "memory");
              } else if (word >= begin && word + 4 <= end) {  // asynchronous: the whole ring in flight
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(word) : "memory");
              } else {  // a word that sticks out of the array, at its first or last token
                uint32_t w = 0;
                for (int b = 0; b < 4; ++b)
                  if (word + b >= begin && word + b < end)
                    w |= (uint32_t)*reinterpret_cast<const uint8_t*>(word + b) << (8 * b);
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(w) : "memory");
              }
            }
          }
          __threadfence_block();
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(q_full + stage))
                       : "memory");
          ++count;
          if (++stage == SQ) { stage = 0; phase ^= 1; }
        }
      }
      if (lane == 0) issued[1] = count;
      asm volatile("cp.async.wait_all;" ::: "memory");  // nothing in flight when the CTA ends
    }
  } else if (warp < 4 + kGroups * kGroupWarps) {
    // ---------------- converters: 16 features of a token at a time.  Eight neighbouring lanes
    // take four 16-byte pieces of rows r and r ^ 5: under the 128-byte swizzle (piece ^ row) of
    // both tiles, neither their loads nor their stores (every other piece) meet in a bank.
    reg_dec<40>();
    const int group = (warp - 4) / kGroupWarps;
    const int tid = (threadIdx.x - 128) % (32 * kGroupWarps);
    const int c = (tid & 3) | (tid >> 1 & 4);   // features 16 c .. 16 c + 15 of the tile
    const int r7 = (tid >> 4 & 3) ^ (tid & 4 ? 5 : 0);
    const int k0 = (tid >> 6) * 8 + r7;         // first token of the stage; the next are 16 apart
    const uint32_t src0 = k0 * BM + ((c ^ r7) << 4);
    const uint32_t dst0 = (c >> 2) * 8192 + k0 * 128 + ((2 * (c & 3) ^ r7) << 4);
    const uint32_t base = smem_u32(smem);
    const uint32_t byte = 0x4440 | c >> 1;      // this thread's scale byte of a token's word
    const uint32_t skew = (uint32_t)reinterpret_cast<uintptr_t>(p.scale);
    int sq = group % SQ, sa = group % SA, sb = group % SB;
    uint32_t pq = 0, pa = 0, pb = 0;
    int skip = group;                           // stages until this group's next
    bool ok = true;
    for (int u = pair; u < units && ok; u += pairs) {
      const Unit t = unit_of<BN>(p, u);
      int kb = t.kb0 + skip;  // (a tile's first scale byte is a multiple of 4 from its row's)
      for (; kb < t.kb1; kb += kGroups) {
        const bool w = wait_bounded(q_full + sq, pq, p.max_spins, abort) &&
                       wait_bounded(a_empty + sa, pa ^ 1, p.max_spins, abort);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        const uint32_t src = base + (SA * A_BYTES + SB * B_BYTES) + sq * Q_BYTES + src0;
        const uint32_t scale = base + (SA * A_BYTES + SB * B_BYTES + SQ * Q_BYTES) + (sq * 2 * BK + k0) * 4;
        const uint32_t dst = base + sa * A_BYTES + dst0;
        uint32_t E[kItems], top = 0;
        uint4 next = lds128(src);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          if (p.scale4) {
            E[i] = __byte_perm(lds32(scale + 64 * i), 0, byte);
          } else {  // the byte after the token's place in its first word
            const uint32_t off = skew + (uint32_t)(kb * BK + k0 + 16 * i) * (uint32_t)p.ld_scale & 3;
            E[i] = __byte_perm(lds32(scale + 64 * i), lds32(scale + 4 * BK + 64 * i), off + (c >> 1)) & 255u;
          }
          top = max(top, E[i]);
        }
        // up to E = 134 the factor 2^(E - 127) 2^120 is one bf16 number; above, two products
        const bool wide = __any_sync(0xffffffffu, top > 134u);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const uint4 raw = next;
          if (i + 1 < kItems) next = lds128(src + (i + 1) * 16 * BM);
          const uint32_t f = wide ? 0x7b807b80u : E[i] * 0x00800080u + 0x3c003c00u;
          uint4 lo, hi;
          e4m3x4_bf16(raw.x, f, lo.x, lo.y);
          e4m3x4_bf16(raw.y, f, lo.z, lo.w);
          e4m3x4_bf16(raw.z, f, hi.x, hi.y);
          e4m3x4_bf16(raw.w, f, hi.z, hi.w);
          if (wide) {  // a marked block is NaN; tokens past the end (no scale) are zeros
            const uint32_t g = E[i] == 255u ? 0x7fc07fc0u : E[i] * 0x00800080u;
            lo.x = bf16x2_mul(lo.x, g); lo.y = bf16x2_mul(lo.y, g);
            lo.z = bf16x2_mul(lo.z, g); lo.w = bf16x2_mul(lo.w, g);
            hi.x = bf16x2_mul(hi.x, g); hi.y = bf16x2_mul(hi.y, g);
            hi.z = bf16x2_mul(hi.z, g); hi.w = bf16x2_mul(hi.w, g);
          }
          sts128(dst + i * 16 * 128, lo);
          sts128((dst ^ 16) + i * 16 * 128, hi);
        }
        fence_proxy_async_smem();
        __syncwarp();
        // the arrival at the issuer says that this CTA's part of D is there, too
        bool there = true;
        if (lane == 0) {
          mbar_arrive(q_empty + sq);
          there = wait_bounded(b_full + sb, pb, p.max_spins, abort);
          if (there) arrive_remote(first_cta(a_full + sa));
        }
        if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
        if ((sb += kGroups) >= SB) { sb -= SB; pb ^= 1; }
        if ((sq += kGroups) >= SQ) { sq -= SQ; pq ^= 1; }
        if ((sa += kGroups) >= SA) { sa -= SA; pa ^= 1; }
      }
      skip = kb - t.kb1;
    }
  } else {
    // ---------------- epilogue: a warp owns 32 features and half of the tile's columns
    reg_inc<152>();
    // TMEM lane to feature: the converters' order 0 2 1 3 of each four
    const int place = (lane & ~3) | ((lane & 1) << 1) | ((lane >> 1) & 1);
    epilogue<BN>(p, reinterpret_cast<float*>(smem + Smem<BN>::epilogue), tmem, tfull, tempty, abort,
                 warp - 4 - kGroups * kGroupWarps, lane, place, rank, pair, pairs);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {  // every role of this CTA has stopped
    if (*abort) {
      if (p.gave_up) p.gave_up[blockIdx.x] = 1;
      land_scaled(q_full, SQ, issued[0], issued[1]);
    }
    if (rank != 0) wait_drain(drain, 0);  // the issuer's arrivals here have come
  }
  __syncwarp();
  cluster_sync();  // neither CTA leaves while the other may still reach its memory
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kCols);
  }
}

// The same product from A already in bf16 (in the workspace): where a feature's tile meets many
// tiles of columns, converting it once and for all costs less than once a tile.  Per CTA
//   warp 0        TMA producer: A (64 tokens x 128 features) and half of the D tile
//   warp 1        MMA issuer (one thread, in the pair's first CTA)
//   warp 2        TMEM allocator
//   warp 3        tells the issuer of each stage that has landed
//   warps 4..11   epilogue
constexpr int RBN = 256, RS = 6;                       // columns of a tile; stages
constexpr int R_STAGE = A_BYTES + BK * RBN;            // A, and half of D's columns
constexpr int RNT = 32 * 12;
constexpr int kRowsEpilogue = RS * R_STAGE + 512;
constexpr int kRowsSmem = 1024 + kRowsEpilogue + 8 * 32 * 9 * 4;
static_assert((3 * RS + 5) * 8 + 16 <= 512 && kRowsSmem <= 227 * 1024, "shared memory");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(RNT, 1)
    k_wgrad_rows(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmD,
                 const WgradP p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RS * R_STAGE);
  uint64_t* empty = full + RS;
  uint64_t* ready = empty + RS;             // used in the first CTA: both CTAs' stages have landed
  uint64_t* tfull = ready + RS;
  uint64_t* tempty = tfull + 2;             // used in the first CTA
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int units = p.whole + p.tail * p.splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < RS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
      mbar_init(ready + s, 2);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tempty + a, 2 * 8);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc_pair(tmem_slot, 2 * RBN);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  grid_trigger();
  if (threadIdx.x == 33 && p.gave_up) p.gave_up[blockIdx.x] = 0;  // as in k_wgrad
  if (warp == 0 && lane == 0) {
    prefetch_map(&tmA);
    prefetch_map(&tmD);
    int stage = 0, count = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = pair; u < units && ok; u += pairs) {
      const Unit t = unit_of<RBN>(p, u);
      for (int kb = t.kb0; kb < t.kb1; ++kb, ++count) {
        if (!wait_bounded(empty + stage, phase ^ 1, p.max_spins, abort)) { ok = false; break; }
        mbar_expect_tx(full + stage, R_STAGE);
        uint8_t* to = smem + stage * R_STAGE;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          tma_load_2d(to + j * 8192, &tmA, full + stage, t.m0 + rank * BM + 64 * j, kb * BK);
          tma_load_2d(to + A_BYTES + j * 8192, &tmD, full + stage, t.n0 + rank * (RBN / 2) + 64 * j, kb * BK);
        }
        if (++stage == RS) { stage = 0; phase ^= 1; }
      }
    }
    wait_landed(full, RS, count);  // whichever role gives up
  } else if (warp == 1 && lane == 0 && rank == 0) {
    constexpr uint32_t idesc = idesc_bf16(PM, RBN, true, true);
    int stage = 0, acc = 0;
    uint32_t phase = 0, pacc = 0;
    bool ok = true;
    for (int u = pair; u < units && ok; u += pairs) {
      const Unit t = unit_of<RBN>(p, u);
      for (int c0 = t.kb0; c0 < t.kb1 && ok; c0 += kChunk) {
        if (!wait_bounded(tempty + acc, pacc ^ 1, p.max_spins, abort)) { ok = false; break; }
        tc_fence_after();
        const int c1 = min(t.kb1, c0 + kChunk);
        for (int kb = c0; kb < c1; ++kb) {
          if (!wait_bounded(ready + stage, phase, p.max_spins, abort)) { ok = false; break; }
          tc_fence_after();
          const uint32_t ab = smem_u32(smem + stage * R_STAGE), bb = ab + A_BYTES;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            mma_pair(tmem + acc * RBN, sw128_desc(ab + k * 2048, 8192, 1024),
                     sw128_desc(bb + k * 2048, 8192, 1024), idesc, ((kb - c0) | k) != 0);
          commit_pair(empty + stage);
          if (++stage == RS) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        commit_pair(tfull + acc);
        acc ^= 1;
        if (acc == 0) pacc ^= 1;
      }
    }
    commit_pair(drain);
    wait_drain(drain, 0);
  } else if (warp == 3 && lane == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = pair; u < units && ok; u += pairs) {
      const Unit t = unit_of<RBN>(p, u);
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        if (!wait_bounded(full + stage, phase, p.max_spins, abort)) { ok = false; break; }
        arrive_remote(first_cta(ready + stage));
        if (++stage == RS) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp >= 4) {
    epilogue<RBN>(p, reinterpret_cast<float*>(smem + kRowsEpilogue), tmem, tfull, tempty, abort, warp - 4,
                  lane, lane, rank, pair, pairs);
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {  // as in k_wgrad (the rank read again: kept over the roles it would spill)
    if (*abort && p.gave_up) p.gave_up[blockIdx.x] = 1;
    if (cluster_rank() != 0) wait_drain(drain, 0);
  }
  __syncwarp();
  cluster_sync();  // neither CTA leaves while the other may still reach its memory
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * RBN);
  }
}

// Adds the split tiles' partial sums in order, into G in either layout: 32 x 32 of a tile, an
// element a thread, so that a small matrix's few blocks have their loads in flight at once.  Where
// a CTA gave up, parts may be missing: then G stays as it was.
__global__ void __launch_bounds__(1024) k_wgrad_join(const WgradP p, int bn) {
  __shared__ float block[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int tile = p.whole + blockIdx.z;
  const int i0 = blockIdx.y * 32, j0 = blockIdx.x * 32;
  const int64_t row0 = (int64_t)(tile % p.tiles_m) * PM + i0, col0 = (int64_t)(tile / p.tiles_m) * bn + j0;
  if (row0 >= p.m || col0 >= p.n) return;
  grid_wait();
  const int missing = threadIdx.x < p.ctas ? p.gave_up[threadIdx.x] : 0;
  const int64_t plane = (int64_t)PM * bn;
  const float* from = p.parts + blockIdx.z * p.splits * plane + (int64_t)(i0 + ty) * bn + j0 + tx;
  float sum = 0.f;
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) sum += from[s * plane];
  if (__syncthreads_or(missing)) return;
  int64_t i = row0 + ty, j = col0 + tx;
  if (!p.transposed) {
    if (i >= p.m || j >= p.n) return;
    float* g = p.out + i * p.ldg + j;
    *g = sum + (p.accumulate ? *g : 0.f);
    return;
  }
  block[ty][tx] = sum;
  __syncthreads();
  i = row0 + tx;
  j = col0 + ty;
  if (i >= p.m || j >= p.n) return;
  float* g = p.out + j * p.ldg + i;
  *g = block[tx][ty] + (p.accumulate ? *g : 0.f);
}

// D into rows that a TMA map can take (a multiple of 8 columns, the rest zero), 8 columns a thread.
template <typename I>
__global__ void __launch_bounds__(256) k_wgrad_pad(const __nv_bfloat16* d, int64_t ldd,
                                                   __nv_bfloat16* out, int64_t ldo, int64_t tokens,
                                                   int64_t n, const RowDiv<I> row_of) {
  const I per_row = (I)(ldo / 8), total = (I)(tokens * per_row);
  const unsigned short* from = reinterpret_cast<const unsigned short*>(d);
  for (I i = (I)blockIdx.x * 256 + threadIdx.x; i < total; i += (I)gridDim.x * 256) {
    const I r = row_of(i);
    const int64_t row = r, col = (int64_t)(i - r * per_row) * 8;
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = col + j < n ? __ldg(from + row * ldd + col + j) : 0u;
    st_vec(out + row * ldo + col, make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16));
  }
}

__global__ void __launch_bounds__(256) k_wgrad_zero(float* G, int64_t ldg, int64_t rows, int64_t cols) {
  const int64_t total = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / cols;
    G[row * ldg + i - row * cols] = 0.f;
  }
}

// ---------------------------------------------------------------- host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// 2-D map of [rows][cols] with rows `stride` bytes apart, box {b0, b1}.
dion_status map2d(CUtensorMap* m, const void* base, CUtensorMapDataType type,
                  CUtensorMapSwizzle swizzle, uint64_t cols, uint64_t rows, uint64_t stride,
                  uint32_t b0, uint32_t b1) {
  const EncodeTiledFn f = encode_fn();
  if (!f) return set_error(DION_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {stride};
  cuuint32_t box[2] = {b0, b1};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = f(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(DION_ERR_CUDA, "cuTensorMapEncodeTiled -> %d (%llu x %llu, stride %llu)", (int)r,
                     (unsigned long long)rows, (unsigned long long)cols, (unsigned long long)stride);
  return DION_OK;
}

#define DION_TRY(call)              \
  do {                              \
    const dion_status st_ = (call); \
    if (st_ != DION_OK) return st_; \
  } while (0)

// Pairs of SMs, and the fewest blocks in a split: below two, a pair's start and the join cost
// more than the tokens.  Plans (and so workspace sizes) do not depend on the device asked.
constexpr int kPairs = 74, kMinBlocks = 2;
constexpr int kMaxCtas = 1024;  // of a launch: k_wgrad_join looks at each with a thread
// What a block of 64 tokens costs a pair, and what parts and their join cost: a launch, and a share
// for each tile and each part, us.  The round is split where the blocks that it saves cost more.
// Split and not: 512 x 1024 x 1024 20.5 and 15.1 us, 1024 x 1024 x 1024 22.1 and 18.5,
// 1536 x 1024 x 1024 22.6 and 22.6, 2048 x 1024 x 1024 23.5 and 26.6, 3000 x 1024 x 1024 25.0 and
// 32.8; 1024 x 256 x 256 14.4 and 18.5.
constexpr double kBlockUs = 0.5, kJoinUs = 3, kJoinTileUs = 0.25, kJoinPartUs = 0.03;
// A is converted beforehand (k_wgrad_rows) from this many columns and tokens on.  Converted first
// and in the kernel, us: 16384 x 4096 x 11008 1026 and 1247, 8192 x 2048 x 2048 63 and 73,
// 1024 x 4096 x 4096 54 and 63, 512 x 4096 x 11008 78 and 92; but 16384 x 4096 x 512 101 and 85,
// 4096 x 1024 x 1024 29 and 27, 200 x 4096 x 4096 46 and 43.
constexpr int64_t kRowsColumns = 1536, kRowsTokens = 512;

struct GradPlan {
  int bn, tiles_m, whole, tail, splits, blocks, blocks_per_split;
  bool pad, rows;       // D is copied into padded rows; A is converted beforehand
  int64_t ldd;          // of the padded copy
  size_t parts_bytes, pad_bytes, rows_bytes;
};

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

GradPlan plan_of(const dion_grad_source& s) {
  GradPlan g{};
  const int64_t m = s.kept.features, n = s.n;
  g.bn = n > 128 ? 256 : 128;
  g.tiles_m = (int)((m + PM - 1) / PM);
  g.blocks = (int)((s.kept.tokens + BK - 1) / BK);
  const int64_t tiles = g.tiles_m * ((n + g.bn - 1) / g.bn);
  const int64_t tail = tiles % kPairs;
  // the last, partial round is split so that it takes 1 / splits of a round
  int64_t want = tail > 0 ? kPairs / tail : 1;
  want = std::min<int64_t>(want, g.blocks / kMinBlocks);
  g.splits = 1;
  if (want > 1) {
    const int per = (int)((g.blocks + want - 1) / want), splits = (g.blocks + per - 1) / per;
    const double join = kJoinUs + kJoinTileUs * tail + kJoinPartUs * tail * splits;
    if ((g.blocks - per) * kBlockUs > join) {
      g.blocks_per_split = per;
      g.splits = splits;
    }
  }
  g.tail = g.splits > 1 ? (int)tail : 0;
  g.whole = (int)(tiles - g.tail);
  g.pad = !rows_aligned16(s.d, s.ldd, 2);
  g.ldd = (n + 7) / 8 * 8;
  // (and behind the parts a word per CTA)
  g.parts_bytes = g.tail > 0 ? (size_t)g.tail * g.splits * PM * g.bn * 4 + 4 * kMaxCtas : 0;
  g.rows = n >= kRowsColumns && s.kept.tokens >= kRowsTokens;
  g.rows_bytes = g.rows ? up256((size_t)s.kept.tokens * kept_ld(m) * 2) : 0;
  g.pad_bytes = g.pad ? up256((size_t)s.kept.tokens * g.ldd * 2) : 0;
  return g;
}

dion_status check_shape(const dion_grad_source& s, int i) {
  DION_TRY(check_tokens(s.kept.tokens));
  const int64_t m = s.kept.features;
  if (m < 1 || m > (1 << 24) || s.n < 1 || s.n > (1 << 24))
    return set_error(DION_ERR_UNSUPPORTED_SHAPE, "source %d: m and n must lie in [1, 2^24]", i);
  if ((m / PM + 1) * (s.n / 128 + 1) > (1 << 30))
    return set_error(DION_ERR_UNSUPPORTED_SHAPE, "source %d: m n is too large", i);
  if (s.kept.tokens > INT32_MAX - BK)
    return set_error(DION_ERR_UNSUPPORTED_SHAPE, "source %d: too many tokens", i);
  return DION_OK;
}

dion_status check_source(const dion_grad_source& s, int i) {
  DION_TRY(check_shape(s, i));
  DION_TRY(check_kept(s.kept));
  if (s.kept.tokens > 0) DION_TRY(check_rows("d", s.d, s.ldd, s.n, 2));
  DION_TRY(check_rows("G", s.G, s.ldg, s.transposed ? s.kept.features : s.n, 4));
  return DION_OK;
}

typedef void (*WgradKernel)(const CUtensorMap, const CUtensorMap, const WgradP);
dion_status launch(WgradKernel kernel, int threads, int smem, const CUtensorMap& ma, const CUtensorMap& md,
                   const WgradP& p, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return set_error(DION_ERR_CUDA, "k_wgrad: %s", cudaGetErrorString(e));
  kernel<<<(unsigned)p.ctas, threads, smem, s>>>(ma, md, p);
  return launch_status("k_wgrad");
}

dion_status one_grad(const dion_grad_source& src, int accumulate, char* ws, int32_t* status,
                     int64_t max_spins, int sms, cudaStream_t s) {
  const int64_t m = src.kept.features, n = src.n, tokens = src.kept.tokens;
  if (tokens == 0) {
    if (accumulate) return DION_OK;
    k_wgrad_zero<<<sms * 4, 256, 0, s>>>(src.G, src.ldg, src.transposed ? n : m, src.transposed ? m : n);
    return launch_status("k_wgrad_zero");
  }
  const GradPlan g = plan_of(src);
  const void* d = src.d;
  int64_t ldd = src.ldd;
  if (g.pad) {
    __nv_bfloat16* copy = reinterpret_cast<__nv_bfloat16*>(ws + up256(g.parts_bytes));
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(src.d);
    if (tokens * (g.ldd / 8) + sms * 8 * 256 < (int64_t(1) << 31))
      k_wgrad_pad<uint32_t><<<sms * 8, 256, 0, s>>>(from, src.ldd, copy, g.ldd, tokens, n, RowDiv<uint32_t>(g.ldd / 8));
    else
      k_wgrad_pad<int64_t><<<sms * 8, 256, 0, s>>>(from, src.ldd, copy, g.ldd, tokens, n, RowDiv<int64_t>(g.ldd / 8));
    DION_TRY(launch_status("k_wgrad_pad"));
    d = copy;
    ldd = g.ldd;
  }
  const int64_t ld = kept_ld(m);
  CUtensorMap mq, md;
  if (g.rows) {
    char* rows = ws + up256(g.parts_bytes) + g.pad_bytes;
    dion_act_kept all = src.kept;
    all.features = ld;  // whole blocks: rows of the copy are aligned
    DION_TRY(dion_act_load(&all, rows, ld, DION_BF16, s));
    DION_TRY(map2d(&mq, rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)ld,
                   (uint64_t)tokens, (uint64_t)ld * 2, 64, BK));
  } else DION_TRY(map2d(&mq, src.kept.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B,
                 (uint64_t)ld, (uint64_t)tokens, (uint64_t)ld, BM, BK));
  DION_TRY(map2d(&md, d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)n,
                 (uint64_t)tokens, (uint64_t)ldd * 2, 64, BK));
  WgradP p{};
  p.scale = src.kept.scale;
  p.out = src.G;
  p.parts = reinterpret_cast<float*>(ws);
  p.status = status;
  p.ctas = 2 * (int)std::min<int64_t>(std::min(sms, kMaxCtas) / 2, g.whole + (int64_t)g.tail * g.splits);
  p.gave_up = g.tail > 0 ? reinterpret_cast<int32_t*>(ws + g.parts_bytes - 4 * kMaxCtas) : nullptr;
  p.tokens = tokens;
  p.ld_scale = ld / DION_ACT_BLOCK;
  p.ldg = src.ldg;
  p.m = m;
  p.n = n;
  p.tiles_m = g.tiles_m;
  p.whole = g.whole;
  p.tail = g.tail;
  p.splits = g.splits;
  p.blocks = g.blocks;
  p.blocks_per_split = g.blocks_per_split;
  p.transposed = src.transposed != 0;
  p.accumulate = accumulate != 0;
  p.vec = aligned_to(src.G, 32) && src.ldg % 8 == 0;
  p.scale4 = p.ld_scale % 4 == 0 && aligned_to(p.scale, 4);
  p.max_spins = max_spins;
  const dion_status st = g.rows        ? launch(k_wgrad_rows, RNT, kRowsSmem, mq, md, p, s)
                         : g.bn == 256 ? launch(k_wgrad<256>, NT, Smem<256>::bytes, mq, md, p, s)
                                       : launch(k_wgrad<128>, NT, Smem<128>::bytes, mq, md, p, s);
  if (st != DION_OK || g.tail == 0) return st;
  return launch_status("k_wgrad_join", launch_after(k_wgrad_join, dim3((unsigned)(g.bn / 32), PM / 32, (unsigned)g.tail),
                                                    1024, 0, s, p, g.bn));
}

}  // namespace

dion_status weight_grad(const dion_grad_source* src, int32_t nsrc, int32_t accumulate, void* ws,
                        size_t ws_bytes, int32_t* d_status, bool clear, int64_t max_spins, void* stream) {
  if (nsrc < 0) return set_error(DION_ERR_INVALID_ARG, "nsources < 0");
  if (nsrc > 0 && !src) return set_error(DION_ERR_INVALID_ARG, "sources is NULL");
  for (int32_t i = 0; i < nsrc; ++i) DION_TRY(check_source(src[i], i));
  const size_t need = dion_weight_grad_workspace(src, nsrc);
  if (need && !ws) return set_error(DION_ERR_INVALID_ARG, "workspace is NULL");
  if (ws_bytes < need)
    return set_error(DION_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  if (need && !aligned_to(ws, 32)) return set_error(DION_ERR_MISALIGNED, "workspace is not 32-byte aligned");
  if (d_status && !aligned_to(d_status, 4))
    return set_error(DION_ERR_MISALIGNED, "d_status is not 4-byte aligned");
  int sms = 0;
  DION_TRY(check_sm100(&sms));
  if (clear && nsrc > 0)
    DION_TRY(launch_status("cudaMemsetAsync", cudaMemsetAsync(d_status, 0, (size_t)nsrc * sizeof(int32_t),
                                                              reinterpret_cast<cudaStream_t>(stream))));
  for (int32_t i = 0; i < nsrc; ++i)
    DION_TRY(one_grad(src[i], accumulate, static_cast<char*>(ws), d_status ? d_status + i : nullptr,
                      max_spins, sms, reinterpret_cast<cudaStream_t>(stream)));
  return DION_OK;
}

}  // namespace dion

extern "C" {

size_t dion_weight_grad_workspace(const dion_grad_source* sources, int32_t nsources) {
  size_t most = 0;
  for (int32_t i = 0; sources && i < nsources; ++i) {
    if (dion::check_shape(sources[i], i) != DION_OK) return 0;
    const dion::GradPlan g = dion::plan_of(sources[i]);
    const size_t b = dion::up256(g.parts_bytes) + g.pad_bytes + g.rows_bytes;
    most = b > most ? b : most;
  }
  return most;
}

dion_status dion_weight_grad(const dion_grad_source* sources, int32_t nsources, int32_t accumulate,
                             void* d_workspace, size_t workspace_bytes, int32_t* d_status,
                             void* stream) {
  return dion::weight_grad(sources, nsources, accumulate, d_workspace, workspace_bytes, d_status,
                           false, dion::kDefaultWaitSpins, stream);
}

}  // extern "C"
