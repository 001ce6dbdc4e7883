// Products of MX 4-bit token rows with MX 4-bit weights, grouped by expert:
//   Z[r, n] = sum_c X[r, c] * W[g(r)][n, c],   rows offsets[g] .. offsets[g+1] of group g,
// plain (Y[o(r)] = s[o(r)] * Z[r]) or SiLU-gated (N = 2F weight rows, gate
// rows first: H[r, f] = silu(Z[r, f]) * Z[r, F + f]).
//
// The codes go to the tensor cores as they are: tcgen05.mma kind::mxf4 with
// block scales multiplies E2M1 elements and E8M0 scales of 32-column blocks
// exactly and accumulates in fp32.  As in the other expert products the weights
// are the M operand (128 rows a tile; gated: 16 gate rows, then the 16 up rows
// of the same features, four times) and the token rows N, so that a group of few rows still
// streams whole weight tiles: at decode sizes the product is bound by reading
// the weights, 17/32 byte per element.
//
// Work decomposition: persistent, one CTA per SM, items (group, token tile,
// weight tile) with the weight tile fastest:
//   warp 0     TMA producer: per K step of 256 the 128 x 128 B weight codes,
//              the BN x 128 B token codes and the weights' 1 KB of scales
//   warp 1     TMEM allocator; copies the step's scales into tensor memory
//              (tcgen05.cp) and issues the step's four MMAs (K = 64 each).
//              The issuing thread comes from elect.sync: with a branch on the
//              lane number the compiler does not know that one thread is
//              active, and issue took 75 cycles an instruction (decode, 128
//              tokens: 341 us; elected: 231 us, the weights' floor)
//   warps 2-   epilogue: four warps, or from 64-row tiles on eight, four to
//              each of the two accumulators (one group took 13 to 18 thousand
//              cycles for 128 x 240 results, twice as long as their MMAs)
//   the rest   token scales, one warp per 128 token rows.  Rows of scale bytes
//              lie anywhere (a group starts at any row), so each is fetched in
//              pieces of 16 bytes (two K steps) asynchronously, kRawDepth
//              pieces ahead, and dealt out to the 512-byte tiles that
//              tcgen05.cp reads, in a ring of their own.  (Fetching 4 bytes
//              at a time by one warp took 1200 cycles a step of 240 rows.)
// Tiles of 240 token rows run on pairs of CTAs (two SMs, tcgen05 cta_group::2,
// M = 256): with one CTA a K step brings 16 KB of weights and 30 KB of token
// rows into shared memory and the MMAs read them all, 730 cycles at 128 bytes a
// cycle against 480 of MMAs.  Each CTA of a pair loads its own 128 weight rows
// and half of the token rows, and its tensor core reads the other half from the
// peer.  The even CTA issues for both: its `full` barriers count both CTAs'
// loads, its commits arrive in both, both epilogues report to its `acc_empty`.
// Scales are not shared: each CTA keeps those of its weight rows and of all
// token rows.
// Weight scales are laid out in tiles once, when the handle is made.
// Every wait is bounded (wait_limit_ns); on timeout the kernel records an
// error, drains what it issued, frees tensor memory and returns.  The odd CTA's
// loads count on the even CTA's barriers, so after an abort in either the even
// CTA waits for the loads of both: it has been told how many steps the odd one
// filled, and closes the phases that only one of them filled.
#include <climits>

#include "elem.cuh"
#include "gemm_common.cuh"
#include "mx4.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kChunk = 16;    // accumulator columns an epilogue warp takes at a time
constexpr int kStageWarpBytes = kChunk * (32 * 2 + 16);  // its staging rows (32-bit results: half of them at a time)
constexpr int kRawDepth = 3;  // 16-byte pieces of a row's scales in flight

template <int BN>
struct CfgMx {
  static constexpr bool PAIR = BN == kMx4PairTile;            // tiles of CTA pairs
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int A_BYTES = kBlockM * 128;               // 128 weight rows x 256 codes
  static constexpr int B_BYTES = BN / CTAS * 128;             // this CTA's token rows x 256 codes
  static constexpr int ROW_TILES = (BN + 127) / 128;          // scale tiles across the token rows
  static constexpr int SFA_BYTES = 2 * kMx4ScaleTile;         // two tiles of 128 columns
  static constexpr int SFB_BYTES = 2 * ROW_TILES * kMx4ScaleTile;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES;
  static constexpr int SF_STAGES = PAIR ? 14 : 4;             // the token scales' ring
  static constexpr int ROW_GROUPS = (BN + 31) / 32;           // groups of 32 token rows
  static constexpr int SCALE_WARPS = (BN + 127) / 128;
  static constexpr int EPI_GROUPS = BN > 32 ? 2 : 1;          // groups of four epilogue warps
  static constexpr int SCALE_WARP0 = kEpilogueWarp0 + 4 * EPI_GROUPS;
  static constexpr int THREADS = 32 * (SCALE_WARP0 + SCALE_WARPS);
  static constexpr int RAW_BYTES = ROW_GROUPS * 32 * 16;      // pieces of all rows
  static constexpr int STAGES_RAW = 190 * 1024 / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 9 ? 9 : STAGES_RAW;
  static constexpr int NACC = 2;
  static constexpr int SFA_COL = NACC * BN;                   // tensor-memory columns of the scales
  static constexpr int SFB_COL = SFA_COL + 2 * 4;
  static constexpr int TMEM_RAW = SFB_COL + 2 * 4 * ROW_TILES;
  static constexpr int TMEM_COLS = TMEM_RAW <= 64 ? 64 : TMEM_RAW <= 128 ? 128 : TMEM_RAW <= 256 ? 256 : 512;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * SF_STAGES + 2 * NACC + 1;
  static constexpr int OUT_BYTES = EPI_GROUPS * 4 * kStageWarpBytes;  // the epilogue warps' staging rows
  static constexpr int TABLE = ROW_GROUPS * 32;               // columns of an item: output rows, then factors
  static constexpr int TABLE_BYTES = EPI_GROUPS * 2 * TABLE * 8;  // of each epilogue group, two by turns
  static constexpr int AUX_BYTES = NUM_BARS * 8 + 128 + (3 * kMaxGroups + 1) * 4;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + SF_STAGES * SFB_BYTES + kRawDepth * RAW_BYTES + OUT_BYTES + TABLE_BYTES +
      AUX_BYTES;
  static_assert(STAGE_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "stages must keep 1024-byte alignment");
  static_assert(STAGES >= 3, "ring too shallow");
  static_assert(TMEM_RAW <= 512, "accumulators and scales exceed tensor memory");
  static_assert(SMEM_BYTES <= 232448, "exceeds shared memory per block");
};

// Instruction descriptor of kind::mxf4: E2M1 operands (code 1 in bits 7-9 and
// 10-12), both K-major, N >> 3 at 17-22, E8M0 scales (bit 23), M >> 4 at
// 24-28, K = 64 (bit 31 clear); the byte of the scale columns where this MMA's
// two blocks start: B's at bits 4-5, A's at bits 29-30.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int sf_byte) {
  return (static_cast<uint32_t>(sf_byte) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(sf_byte) << 29);
}

template <bool PAIR>
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptor of a scale tile: 32 rows of 16 bytes, no swizzle,
// 128 bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(128u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  return d;
}

// A scale tile into four tensor-memory columns (the 32 rows repeated in every
// quarter of the lanes); in order with the MMAs of the same thread.  PAIR: in
// both CTAs, each from its own shared memory.
template <bool PAIR>
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t s_desc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(s_desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(s_desc) : "memory");
}

// Tile loads in 2, 3 and 5 dimensions, their bytes counted on `bar` (an address
// in the cluster: PAIR loads of the odd CTA count on the even CTA's barrier).
// The five-dimensional box is the gated one: 4 blocks of 16 gate and the 16 up
// rows, from block c1 of group c2.
#define MOE_TMA_LOAD(DIM, GROUP, COORDS, ...)                                                                       \
  asm volatile("cp.async.bulk.tensor." DIM ".shared::cta.global.tile.mbarrier::complete_tx::bytes" GROUP            \
               ".L2::cache_hint [%0], [%1, " COORDS "], [%2], %3;" ::"r"(smem_u32(dst)),                            \
               "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "l"(policy), __VA_ARGS__                             \
               : "memory")
template <bool PAIR>
__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                        uint64_t policy) {
  if constexpr (PAIR)
    MOE_TMA_LOAD("2d", ".cta_group::2", "{%4, %5}", "r"(c0), "r"(c1));
  else
    MOE_TMA_LOAD("2d", "", "{%4, %5}", "r"(c0), "r"(c1));
}
template <bool PAIR>
__device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                        uint64_t policy) {
  if constexpr (PAIR)
    MOE_TMA_LOAD("3d", ".cta_group::2", "{%4, %5, %6}", "r"(c0), "r"(c1), "r"(c2));
  else
    MOE_TMA_LOAD("3d", "", "{%4, %5, %6}", "r"(c0), "r"(c1), "r"(c2));
}
template <bool PAIR>
__device__ __forceinline__ void load_5d(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                        uint64_t policy) {
  if constexpr (PAIR)
    MOE_TMA_LOAD("5d", ".cta_group::2", "{%4, %7, %7, %5, %6}", "r"(c0), "r"(c1), "r"(c2), "r"(0));
  else
    MOE_TMA_LOAD("5d", "", "{%4, %7, %7, %5, %6}", "r"(c0), "r"(c1), "r"(c2), "r"(0));
}
#undef MOE_TMA_LOAD

// Waits and arrivals across a pair carry cluster scope.
template <bool PAIR>
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
  if constexpr (!PAIR) return mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait that also gives up as soon as another role of the CTA has aborted.
template <bool PAIR>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
  if (try_wait<PAIR>(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  uint32_t spins = 0;
  while (true) {
    if (try_wait<PAIR>(bar, parity)) return true;
    if ((++spins & 15u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > limit_ns) return false;
    }
  }
}
// Arrive on the barrier at this offset in the CTA that issues the MMAs, once
// this warp has read its accumulator (ordered by the tcgen05 fence).
template <bool PAIR>
__device__ __forceinline__ void arrive_issuer(uint64_t* bar) {
  if constexpr (PAIR)
    mbar_arrive_cluster(mapa_shared(smem_u32(bar), 0));
  else
    mbar_arrive(bar);
}
template <bool PAIR>
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  if constexpr (PAIR)
    tc_commit_pair_multicast(bar, 0x3);
  else
    tc_commit(bar);
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// 16 or 4 bytes to shared memory, asynchronously; zeros past `bytes`.
__device__ __forceinline__ void copy16_async(uint32_t saddr, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(saddr), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy4_async(uint32_t saddr, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(saddr), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// To the other CTA's shared memory, at the same offset as p.
__device__ __forceinline__ void store_peer(uint32_t peer, volatile void* p, uint64_t v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(mapa_shared(smem_u32(const_cast<const void*>(p)), peer)), "l"(v)
               : "memory");
}
// Takes `bytes` off what the barrier's phase still expects.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// Parity of the last phase of stage s that a filler at (stage, phase) has filled;
// for a stage not filled yet, of the phase before its first, which has passed.
__device__ __forceinline__ uint32_t ring_parity(uint32_t s, uint32_t stage, uint32_t phase) {
  return s < stage ? phase : phase ^ 1u;
}
// How often stage s of a ring has been filled after `steps` steps.
__device__ __forceinline__ uint64_t fills_of(uint64_t steps, int s, int stages) {
  return (steps + stages - 1 - s) / stages;
}
// One thread of a converged warp, as the compiler knows.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// The groups' rows and token tiles from the offsets, by one warp.  Offsets are
// held to [0, rows] and a group that ends before it starts has no rows, so
// whatever they hold no access leaves the buffers.
__device__ __forceinline__ void build_groups(const int* offsets, int G, int rows, int tile, int* tile_start,
                                             int* g_row0, int* g_rows, int lane) {
  constexpr int kRuns = 10;  // of 32 groups, their offsets loaded together (one load latency for 320 groups)
  int carry = 0;
  for (int g0 = 0; g0 < G; g0 += 32 * kRuns) {
    int lo[kRuns], hi[kRuns];
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      const int g = g0 + 32 * j + lane;
      lo[j] = g < G ? __ldg(offsets + g) : 0;
      hi[j] = g < G ? __ldg(offsets + g + 1) : 0;
    }
#pragma unroll
    for (int j = 0; j < kRuns; ++j) {
      if (g0 + 32 * j >= G) break;
      const int g = g0 + 32 * j + lane;
      const int first = min(max(lo[j], 0), rows);
      const int n = max(min(max(hi[j], 0), rows) - first, 0);
      const int tiles = (n + tile - 1) / tile;
      int incl = tiles;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      if (g < G) {
        g_row0[g] = first;
        g_rows[g] = n;
        tile_start[g] = carry + incl - tiles;
      }
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (lane == 0) tile_start[G] = carry;
}

// ---------------------------------------------------------------- epilogue --
// A chunk is 16 accumulator columns (token rows) of the 32 tensor-memory lanes
// of one warp, loaded in the 16x256b shape: of each half of 16 lanes, register
// 4j + 2h + i of lane l holds lane (l / 4) + 8h, column 8j + 2 (l % 4) + i.

__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, float (&r)[8]) {
  uint32_t u[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(u[i]);
}

// One chunk: lanes 0-15 in lo (gated: gate values), lanes 16-31 in hi (the up
// values of the same features).
struct Chunk {
  float lo[8], hi[8];
};
__device__ __forceinline__ void load_chunk(uint32_t taddr, int c0, Chunk& c) {
  tmem_ld_16x256b_x2(taddr + c0, c.lo);
  tmem_ld_16x256b_x2(taddr + (16u << 16) + c0, c.hi);
}
// Completes the loads in flight; no use of the registers moves before it.
__device__ __forceinline__ void wait_chunk(Chunk& c) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(c.lo[0]), "+f"(c.lo[1]), "+f"(c.lo[2]), "+f"(c.lo[3]), "+f"(c.lo[4]), "+f"(c.lo[5]), "+f"(c.lo[6]),
                 "+f"(c.lo[7]), "+f"(c.hi[0]), "+f"(c.hi[1]), "+f"(c.hi[2]), "+f"(c.hi[3]), "+f"(c.hi[4]),
                 "+f"(c.hi[5]), "+f"(c.hi[6]), "+f"(c.hi[7])
               :
               : "memory");
}

// Four 8 x 8 blocks of 16-bit values to shared memory, transposed: lane 8k + j
// gives the address of column j of block k.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t saddr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<bf16>(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 t = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// Results of one chunk, 16 product rows of FEATS features, to the warp's staging
// rows in shared memory and from there to the output in 16-byte pieces: a
// thread holds one feature of several product rows, the output wants a row's
// features together.  Staging rows are 16 bytes longer than their features,
// which keeps the transposed stores and the row loads free of bank conflicts.
// 32-bit results go eight rows at a time (half j of the chunk).
template <typename T, int FEATS>
struct Stage {
  static constexpr int PITCH = FEATS * static_cast<int>(sizeof(T)) + 16;
  static constexpr int PIECES = FEATS * static_cast<int>(sizeof(T)) / 16;  // per row
  static constexpr int ROUNDS = sizeof(T) == 4 ? 2 : 1;
  static constexpr int ROWS = kChunk / ROUNDS;
  static_assert(ROWS * PITCH <= kStageWarpBytes, "staging rows");
};

// v: FEATS / 16 groups of 16 features, group g register 4j + 2h + i as in a chunk.
template <typename T, int FEATS>
__device__ __forceinline__ void stage_rows(uint32_t sbase, const float* v, int j, int lane) {
  constexpr int PITCH = Stage<T, FEATS>::PITCH;
#pragma unroll
  for (int g = 0; g < FEATS / 16; ++g) {
    const float* r = v + 8 * g;
    if constexpr (sizeof(T) == 2) {
      // blocks: (rows 0-7, features 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
      const uint32_t p[4] = {pack2<T>(r[0], r[1]), pack2<T>(r[2], r[3]), pack2<T>(r[4], r[5]), pack2<T>(r[6], r[7])};
      const int block = lane >> 3, row = (block >> 1) * 8 + (lane & 7);
      stmatrix_x4_trans(sbase + row * PITCH + (16 * g + (block & 1) * 8) * 2, p);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 2 * (lane & 3) + (k & 1), feat = 16 * g + (lane >> 2) + (k >> 1) * 8;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + row * PITCH + feat * 4), "f"(r[4 * j + k]) : "memory");
      }
    }
  }
}

// Staged rows to out[orow[row]][feat0 ...] (negative: none).  vec: output rows
// are whole 16-byte pieces.
template <typename T, int FEATS>
__device__ __forceinline__ void store_rows(const Mx4GemmArgs& a, uint32_t sbase, const int* orow, int feat0, bool vec,
                                           int lane) {
  using St = Stage<T, FEATS>;
  constexpr int PER = 16 / sizeof(T);
  constexpr int N = (St::ROWS * St::PIECES + 31) / 32;
  const int piece = lane % St::PIECES, feat = feat0 + piece * PER;
  // all shared loads, then all stores: no branch between them
  uint4 w[N];
  int o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = (32 * i + lane) / St::PIECES;
    o[i] = orow[row % St::ROWS];
    if (32 * i + 31 >= St::ROWS * St::PIECES && row >= St::ROWS) o[i] = -1;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                 : "r"(sbase + (row % St::ROWS) * St::PITCH + piece * 16));
  }
  T* const out = static_cast<T*>(a.out) + feat;
  if (vec) {
    const bool in = feat < a.out_cols;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in && o[i] >= 0) *reinterpret_cast<uint4*>(out + static_cast<size_t>(o[i]) * a.out_cols) = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const T* e = reinterpret_cast<const T*>(&w[i]);
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (o[i] >= 0 && feat + k < a.out_cols) out[static_cast<size_t>(o[i]) * a.out_cols + k] = e[k];
    }
  }
}

// silu(gate) * up.  32-bit results: by the full exponential, of -|gate| so that
// neither end overflows, within 7 half steps.  16-bit results: by the approximate
// one (2 + |gate| steps of 2^-22, 0 below a gate of -87), which their own rounding
// covers; the epilogue of a prompt's product is bound by its instructions.
template <typename T>
__device__ __forceinline__ float silu_up(float gate, float up) {
  if constexpr (sizeof(T) == 4) {
    const float e = expf(-fabsf(gate)), r = __frcp_rn(1.0f + e);
    return gate * (gate < 0.f ? e * r : r) * up;
  }
  return gate * sigmoid_approx(gate) * up;
}

// One chunk of results: SiLU gate, the rows' factors, staging and stores.
template <bool GATED, typename T>
__device__ __forceinline__ void finish_chunk(const Mx4GemmArgs& a, const Chunk& c, uint32_t sbase, const int* orow,
                                             const float* factor, int feat0, bool vec, int lane) {
  constexpr int FEATS = GATED ? 16 : 32;
  float v[FEATS / 2];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = GATED ? silu_up<T>(c.lo[k], c.hi[k]) : c.lo[k];
    if (!GATED) v[(8 + k) % (FEATS / 2)] = c.hi[k];
  }
  if (a.row_scale != nullptr) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 f = *reinterpret_cast<const float2*>(factor + 8 * j + 2 * (lane & 3));
#pragma unroll
      for (int g = 0; g < FEATS / 16; ++g) {
        v[8 * g + 4 * j] *= f.x;
        v[8 * g + 4 * j + 1] *= f.y;
        v[8 * g + 4 * j + 2] *= f.x;
        v[8 * g + 4 * j + 3] *= f.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < Stage<T, FEATS>::ROUNDS; ++j) {
    __syncwarp();  // what was staged before has been read
    stage_rows<T, FEATS>(sbase, v, j, lane);
    __syncwarp();
    store_rows<T, FEATS>(a, sbase, orow + j * Stage<T, FEATS>::ROWS, feat0, vec, lane);
  }
}

template <bool GATED>
__device__ __forceinline__ void finish_any(const Mx4GemmArgs& a, const Chunk& c, uint32_t sbase, const int* orow,
                                           const float* factor, int feat0, int lane) {
  switch (a.out_type) {
    case kBf16: finish_chunk<GATED, bf16>(a, c, sbase, orow, factor, feat0, a.out_wide, lane); break;
    case kFp16: finish_chunk<GATED, __half>(a, c, sbase, orow, factor, feat0, a.out_wide, lane); break;
    default: finish_chunk<GATED, float>(a, c, sbase, orow, factor, feat0, a.out_wide, lane); break;
  }
}

// The valid columns of an item's accumulator (tensor memory at taddr, this
// warp's lanes), the next chunk's load in flight while one is finished;
// release() once all are loaded.  orow and factor: the columns' output rows and
// factors.
template <bool GATED, int BN, typename T, typename Release>
__device__ __forceinline__ void epilogue_typed(const Mx4GemmArgs& a, uint32_t taddr, int feat0, int valid,
                                               const int* orow, const float* factor, uint32_t sbase, int lane,
                                               const Release& release) {
  const bool vec = a.out_wide;
  Chunk even, odd;
  load_chunk(taddr, 0, even);
  // not unrolled: straight-line code for all chunks runs at the rate it is
  // fetched at (8192 tokens' down product: 436 us unrolled)
#pragma unroll 1
  for (int c0 = 0; c0 < valid; c0 += 2 * kChunk) {
    wait_chunk(even);
    const bool more_odd = c0 + kChunk < valid;
    if (more_odd)
      load_chunk(taddr, c0 + kChunk, odd);
    else
      release();
    finish_chunk<GATED, T>(a, even, sbase, orow + c0, factor + c0, feat0, vec, lane);
    if (!more_odd) break;
    wait_chunk(odd);
    if (c0 + 2 * kChunk < valid)
      load_chunk(taddr, c0 + 2 * kChunk, even);
    else
      release();
    finish_chunk<GATED, T>(a, odd, sbase, orow + c0 + kChunk, factor + c0 + kChunk, feat0, vec, lane);
  }
}

template <bool GATED, int BN, typename Release>
__device__ __forceinline__ void epilogue_mx(const Mx4GemmArgs& a, uint32_t taddr, int feat0, int valid,
                                            const int* orow, const float* factor, uint32_t sbase, int lane,
                                            const Release& release) {
  switch (a.out_type) {
    case kBf16: epilogue_typed<GATED, BN, bf16>(a, taddr, feat0, valid, orow, factor, sbase, lane, release); break;
    case kFp16: epilogue_typed<GATED, BN, __half>(a, taddr, feat0, valid, orow, factor, sbase, lane, release); break;
    default: epilogue_typed<GATED, BN, float>(a, taddr, feat0, valid, orow, factor, sbase, lane, release); break;
  }
}

// K split.  A part's chunk is 4 float4 of each lane, stored lane by lane:
// part[slot][warp][chunk][4][32] float4.
template <int BN>
__device__ __forceinline__ float4* part_at(float* part, int slot, int q, int chunk, int lane) {
  return reinterpret_cast<float4*>(part) + (((static_cast<size_t>(slot) * 4 + q) * (BN / kChunk) + chunk) * 4) * 32 + lane;
}
template <int BN>
__device__ __forceinline__ void store_part(float* part, int slot, int q, int chunk, int lane, const Chunk& c) {
  float4* p = part_at<BN>(part, slot, q, chunk, lane);
  __stcg(p, make_float4(c.lo[0], c.lo[1], c.lo[2], c.lo[3]));
  __stcg(p + 32, make_float4(c.lo[4], c.lo[5], c.lo[6], c.lo[7]));
  __stcg(p + 64, make_float4(c.hi[0], c.hi[1], c.hi[2], c.hi[3]));
  __stcg(p + 96, make_float4(c.hi[4], c.hi[5], c.hi[6], c.hi[7]));
}
// Sum of a unit's parts in part order; `own` is the part in c already (or -1).
template <int BN>
__device__ __forceinline__ void sum_parts(float* part, const UnitCursor& cur, const WorkUnit& u, int own, int q,
                                          int chunk, int lane, Chunk& c) {
  float4 f[kMaxGemmKSplit][4];
#pragma unroll
  for (int p = 0; p < kMaxGemmKSplit; ++p) {
    const bool read = p < u.parts && p != own;
    const float4* src = part_at<BN>(part, cur.part_slot(u, p < u.parts ? p : 0), q, chunk, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[p][j] = read ? __ldcg(src + 32 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (p == own) {
      f[p][0] = make_float4(c.lo[0], c.lo[1], c.lo[2], c.lo[3]);
      f[p][1] = make_float4(c.lo[4], c.lo[5], c.lo[6], c.lo[7]);
      f[p][2] = make_float4(c.hi[0], c.hi[1], c.hi[2], c.hi[3]);
      f[p][3] = make_float4(c.hi[4], c.hi[5], c.hi[6], c.hi[7]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 t = f[0][j];
#pragma unroll
    for (int p = 1; p < kMaxGemmKSplit; ++p) {
      t.x += f[p][j].x;
      t.y += f[p][j].y;
      t.z += f[p][j].z;
      t.w += f[p][j].w;
    }
    float* d = j < 2 ? c.lo + 4 * j : c.hi + 4 * (j - 2);
    d[0] = t.x;
    d[1] = t.y;
    d[2] = t.z;
    d[3] = t.w;
  }
}

template <bool GATED, int BN>
__device__ __forceinline__ void mx4_gemm_body(const CUtensorMap& map_w, const CUtensorMap& map_s,
                                              const CUtensorMap& map_x, const Mx4GemmArgs& args) {
  using C = CfgMx<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* sf_ring = ring + C::STAGES * C::STAGE_BYTES;
  uint8_t* raw_scales = sf_ring + C::SF_STAGES * C::SFB_BYTES;
  uint8_t* out_rows = raw_scales + kRawDepth * C::RAW_BYTES;
  int* tables = reinterpret_cast<int*>(out_rows + C::OUT_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(out_rows + C::OUT_BYTES + C::TABLE_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = full + C::STAGES;
  uint64_t* sf_full = empty + C::STAGES;
  uint64_t* sf_empty = sf_full + C::SF_STAGES;
  uint64_t* acc_full = sf_empty + C::SF_STAGES;
  uint64_t* acc_empty = acc_full + C::NACC;
  uint64_t* drain = acc_empty + C::NACC;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* s_last = reinterpret_cast<volatile int*>(tmem_holder + 2);
  volatile int* s_ok = reinterpret_cast<volatile int*>(tmem_holder + 4);  // [group][2 parities][4 warps]
  // pairs, written by the other CTA at its end: whether it aborted, and (from the odd CTA) the steps it loaded
  volatile uint64_t* peer_abort = reinterpret_cast<volatile uint64_t*>(tmem_holder + 24);
  volatile uint64_t* peer_steps = peer_abort + 1;
  volatile uint64_t* own_steps = peer_abort + 2;  // the even CTA's
  int* tile_start = reinterpret_cast<int*>(tmem_holder + 32);
  int* g_row0 = tile_start + kMaxGroups + 1;
  int* g_rows = g_row0 + kMaxGroups;

  constexpr bool PAIR = C::PAIR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = args.G;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;  // 0 issues the MMAs
  // weight tiles of an item: one, or two of a pair (this CTA's: rank)
  const int m_items = (args.m_tiles + C::CTAS - 1) / C::CTAS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::SF_STAGES; ++s) {
      mbar_init(&sf_full[s], C::SCALE_WARPS + (PAIR && rank == 0 ? 1 : 0));
      mbar_init(&sf_empty[s], 1);
    }
    for (int a = 0; a < C::NACC; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], C::CTAS * 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *peer_abort = *peer_steps = *own_steps = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_w);
    tma_prefetch_desc(&map_s);
    tma_prefetch_desc(&map_x);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_holder, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  pdl_wait();  // offsets, rows and outputs belong to earlier work in the stream until here
  if (warp == kEpilogueWarp0) build_groups(args.offsets, G, args.rows, BN, tile_start, g_row0, g_rows, lane);
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();  // both CTAs' barriers are there before any arrival from the peer
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // the host refuses calls of so many items, but groups that overlap may have more
  const long long all_items = static_cast<long long>(tile_start[G]) * m_items;
  const int n_items = all_items > INT_MAX ? 0 : static_cast<int>(all_items);
  if (all_items > INT_MAX && threadIdx.x == 0) atomicOr(args.err, kErrBounds);
  const int mode = BN <= 32 && args.balanced ? kBalanced : kWhole;
  const uint64_t limit = args.wait_limit_ns;
  auto start = [&](UnitCursor& cur) {
    cur.init(mode, n_items, args.k_steps, kMaxGemmKSplit);
    if (PAIR) {  // whole items, dealt out to the pairs
      cur.stride = static_cast<int>(gridDim.x) / 2;
      cur.pos = static_cast<int>(blockIdx.x) / 2;
    }
  };
  auto decode = [&](int item) {
    Item it = decode_item(item, m_items, tile_start, G, n_items, 0);
    it.m = it.m * C::CTAS + rank;
    return it;
  };

  if (warp == 0) {
    if (elect_one()) {
      // ---------------------------------------------------------- producer --
      // weights: streamed once, but by pairs often for two tiles of a group (8192
      // tokens' down product 287 us if streamed past L2, 282 kept)
      const uint64_t pol_w = PAIR ? policy_evict_normal() : policy_evict_first();
      const uint64_t pol_act = policy_evict_last();  // token rows: re-read by the other weight tiles
      UnitCursor cur;
      start(cur);
      WorkUnit u;
      uint32_t stage = 0, phase = 0;
      uint64_t issued = 0;  // K steps (pairs)
      bool ok = true;
      while (ok && !*abort_flag && cur.next(u)) {
        const Item it = decode(u.item);
        const int row_w = it.m * (GATED ? kBlockM / 2 : kBlockM);
        // the pair MMA takes half of its N token rows from each CTA
        const int row_x = g_row0[it.g] + it.n * BN +
                          (PAIR ? rank * (mma_width(g_rows[it.g] - it.n * BN, 16, BN) / 2) : 0);
        const int sfa = (it.g * args.m_stride + it.m) * args.k_steps;  // the tile's first row of map_s
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!wait_bar<PAIR>(&empty[stage], phase ^ 1u, limit, abort_flag)) {
            record_abort(abort_flag, args.err);
            ok = false;
            break;
          }
          uint8_t* st = ring + stage * C::STAGE_BYTES;
          const uint32_t bar = PAIR ? mapa_shared(smem_u32(&full[stage]), 0) : smem_u32(&full[stage]);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::CTAS * (C::A_BYTES + C::B_BYTES + C::SFA_BYTES));
          if (GATED && args.gated_boxes == 1) {
            load_5d<PAIR>(st, &map_w, bar, kb * 128, row_w / 16, it.g, pol_w);
          } else if (GATED) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              load_3d<PAIR>(st + b * 4096, &map_w, bar, kb * 128, row_w + 16 * b, it.g, pol_w);
              load_3d<PAIR>(st + b * 4096 + 2048, &map_w, bar, kb * 128, args.N / 2 + row_w + 16 * b, it.g, pol_w);
            }
          } else {
            load_3d<PAIR>(st, &map_w, bar, kb * 128, row_w, it.g, pol_w);
          }
          load_2d<PAIR>(st + C::A_BYTES, &map_x, bar, kb * 128, row_x, pol_act);
          load_2d<PAIR>(st + C::A_BYTES + C::B_BYTES, &map_s, bar, 0, sfa + kb, pol_w);
          if (PAIR) ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // The loads into each stage must have landed before this CTA may exit (they
      // always complete; the wait is bounded anyway).  A pair's have, since the
      // issuer waits for all; after an abort, see the end.
      for (int s = 0; !PAIR && s < C::STAGES; ++s) mbar_wait(&full[s], ring_parity(s, stage, phase), kDrainLimitNs);
      // The odd CTA stays until the issuer's last reports have reached it.
      for (int s = 0; PAIR && rank == 1 && ok && s < C::STAGES; ++s)
        if (!wait_or_abort(&empty[s], ring_parity(s, stage, phase), limit, abort_flag)) {
          record_abort(abort_flag, args.err);
          ok = false;
        }
      if constexpr (PAIR) {
        if (rank == 0)
          *own_steps = issued;
        else
          store_peer(0, peer_steps, issued);
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // --------------------------------------------------------------- MMA --
      UnitCursor cur;
      start(cur);
      WorkUnit u;
      uint32_t stage = 0, phase = 0, sf_stage = 0, sf_phase = 0, acc = 0, acc_phase = 0;
      bool issued_any = false, ok = true;
      const int mmas = (args.blocks + 1) / 2;  // K = 64 instructions of a whole row
      while (ok && !*abort_flag && cur.next(u)) {
        const Item it = decode(u.item);
        const int width = mma_width(g_rows[it.g] - it.n * BN, 16, BN);
        const uint32_t idesc0 = idesc_mxf4(C::CTAS * kBlockM, width, 0),
                       idesc1 = idesc_mxf4(C::CTAS * kBlockM, width, 2);
        if (!wait_bar<PAIR>(&acc_empty[acc], acc_phase ^ 1u, limit, abort_flag)) {
          record_abort(abort_flag, args.err);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!wait_bar<PAIR>(&sf_full[sf_stage], sf_phase, limit, abort_flag) ||
              !wait_bar<PAIR>(&full[stage], phase, limit, abort_flag)) {
            record_abort(abort_flag, args.err);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(ring + stage * C::STAGE_BYTES);
          const uint64_t a = smem_desc_sw128(st);
          const uint64_t b = smem_desc_sw128(st + C::A_BYTES);
          const uint32_t sfa = st + C::A_BYTES + C::B_BYTES, sfb = smem_u32(sf_ring + sf_stage * C::SFB_BYTES);
          const uint32_t ta = tmem_base + C::SFA_COL, tb = tmem_base + C::SFB_COL;
          const int todo = mmas - kb * 4;  // instructions left in the row: at most 4 in this step
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            tc_copy_scales<PAIR>(ta + 4 * t, smem_desc_scales(sfa + t * kMx4ScaleTile));
#pragma unroll
            for (int j = 0; j < C::ROW_TILES; ++j)
              tc_copy_scales<PAIR>(tb + 4 * (t * C::ROW_TILES + j),
                             smem_desc_scales(sfb + (t * C::ROW_TILES + j) * kMx4ScaleTile));
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // +32 B along K = +2 in the address field
            if (kk < todo)
              tc_mma_mxf4<PAIR>(d_tmem, a + 2 * kk, b + 2 * kk, (kk & 1) ? idesc1 : idesc0, ta + 4 * (kk >> 1),
                          tb + 4 * (kk >> 1) * C::ROW_TILES, (kb > u.kb0 || kk > 0) ? 1u : 0u);
          issued_any = true;
          commit_both<PAIR>(&empty[stage]);
          commit_both<PAIR>(&sf_empty[sf_stage]);
          if (++sf_stage == C::SF_STAGES) {
            sf_stage = 0;
            sf_phase ^= 1u;
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit_both<PAIR>(&acc_full[acc]);
        if (++acc == C::NACC) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (issued_any) {
        // every MMA of this CTA has finished before tensor memory is freed
        if constexpr (PAIR)
          tc_commit_pair(drain);
        else
          tc_commit(drain);
        mbar_wait(drain, 0, kDrainLimitNs);
      }
    }
    if (PAIR && rank == 1 && elect_one()) {
      // -------------------------------------------- relay of the odd CTA --
      // reports this CTA's finished token scales to the issuing CTA.  A fence at
      // cluster scope takes about 2000 cycles on a busy SM, so one covers all
      // steps that are ready, and a thread of its own waits for it (by a fence
      // for each step 8192 tokens' gate/up product took 950 us).
      UnitCursor cur;
      start(cur);
      WorkUnit u;
      long steps = 0;
      while (cur.next(u)) steps += u.kb1 - u.kb0;
      uint32_t sf_stage = 0, sf_phase = 0, out_stage = 0;
      while (steps > 0 && !*abort_flag) {
        if (!wait_bar<PAIR>(&sf_full[sf_stage], sf_phase, limit, abort_flag)) {
          record_abort(abort_flag, args.err);
          break;
        }
        int ready = 0;
        do {
          ++ready;
          if (++sf_stage == C::SF_STAGES) {
            sf_stage = 0;
            sf_phase ^= 1u;
          }
        } while (ready < steps && ready < C::SF_STAGES && try_wait<PAIR>(&sf_full[sf_stage], sf_phase));
        steps -= ready;
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        for (; ready > 0; --ready) {
          asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                           mapa_shared(smem_u32(&sf_full[out_stage]), 0))
                       : "memory");
          if (++out_stage == C::SF_STAGES) out_stage = 0;
        }
      }
      // as the producer does: the issuer's reports on the scales (in the scale warps
      // this wait made the whole kernel 1 % slower)
      for (int s = 0; steps == 0 && s < C::SF_STAGES; ++s)
        if (!wait_or_abort(&sf_empty[s], ring_parity(s, sf_stage, sf_phase), limit, abort_flag)) {
          record_abort(abort_flag, args.err);
          break;
        }
    }
  } else if (warp >= C::SCALE_WARP0) {
    // ------------------------------------------------------- token scales --
    const int w = warp - C::SCALE_WARP0;
    constexpr int GROUPS = (C::ROW_GROUPS + C::SCALE_WARPS - 1) / C::SCALE_WARPS;  // groups of 32 rows of this warp
    const bool wide = args.scales_wide;
    // the scale bytes past a row's last block are taken as zero
    const int full_words = args.blocks >> 2, tail = args.blocks & 3;
    // Pieces are fetched (fetch) kRawDepth ahead of being dealt out (deal);
    // each lane deals out what it fetched itself.
    UnitCursor cur;
    start(cur);
    WorkUnit u;
    u.kb0 = u.kb1 = 0;
    int kb = 0;                                       // the next step to fetch
    int row_x = 0, valid = 0;
    int from[kRawDepth], to[kRawDepth];               // K steps of the pieces in flight: [from, to), both of one pair
    uint32_t stage = 0, phase = 0;
    bool more = true, ok = true;
    auto fetch = [&](int slot) {
      from[slot] = to[slot] = 0;
      if (more && kb >= u.kb1) {
        more = cur.next(u);
        if (more) {
          const Item it = decode(u.item);
          row_x = g_row0[it.g] + it.n * BN;
          valid = min(BN, g_rows[it.g] - it.n * BN);
          kb = u.kb0;
        }
      }
      if (more) {
        from[slot] = kb;
        to[slot] = min(u.kb1, (kb | 1) + 1);
        const int byte = (kb >> 1) * 16;              // of the row
        const int have = args.scale_ld - byte;        // > 0
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
          const int r = 32 * (w * GROUPS + i) + lane;
          const uint32_t dst = smem_u32(raw_scales) + slot * C::RAW_BYTES + r * 16;
          if (w * GROUPS + i >= C::ROW_GROUPS) break;
          const bool in = r < valid;
          const uint8_t* src = args.scales + static_cast<size_t>(row_x + (in ? r : 0)) * args.scale_ld + byte;
          if (wide) {
            copy16_async(dst, src, in ? 16u : 0u);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) copy4_async(dst + 4 * k, src + (4 * k < have ? 4 * k : 0), in && 4 * k < have ? 4u : 0u);
          }
        }
        kb = to[slot];
      }
      copy_commit();
    };
#pragma unroll
    for (int d = 0; d < kRawDepth; ++d) fetch(d);
    while (ok && !*abort_flag && from[0] < to[0]) {
#pragma unroll
      for (int d = 0; d < kRawDepth; ++d) {
        if (!ok || from[d] >= to[d]) break;
        copy_wait<kRawDepth - 1>();
        uint4 piece[GROUPS];
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
          if (w * GROUPS + i >= C::ROW_GROUPS) break;
          const uint32_t src = smem_u32(raw_scales) + d * C::RAW_BYTES + (32 * (w * GROUPS + i) + lane) * 16;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(piece[i].x), "=r"(piece[i].y), "=r"(piece[i].z), "=r"(piece[i].w)
                       : "r"(src));
        }
        for (int step = from[d]; step < to[d]; ++step) {
          ok = __all_sync(0xffffffffu, wait_bar<PAIR>(&sf_empty[stage], phase ^ 1u, limit, abort_flag));
          if (!ok) {
            if (lane == 0) record_abort(abort_flag, args.err);
            break;
          }
          const uint32_t sfb = smem_u32(sf_ring + stage * C::SFB_BYTES);
#pragma unroll
          for (int i = 0; i < GROUPS; ++i) {
            const int g = w * GROUPS + i;
            if (g >= C::ROW_GROUPS) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              uint32_t v = (step & 1) ? (t ? piece[i].w : piece[i].z) : (t ? piece[i].y : piece[i].x);
              const int word = 2 * step + t;
              if (word >= full_words) v = word > full_words || tail == 0 ? 0u : v & ((1u << (8 * tail)) - 1u);
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(sfb + (t * C::ROW_TILES + (g >> 2)) * kMx4ScaleTile +
                                                           lane * 16 + (g & 3) * 4),
                           "r"(v)
                           : "memory");
            }
          }
          fence_async_proxy();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sf_full[stage]);
          if (++stage == C::SF_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) fetch(d);
      }
    }
    copy_wait<0>();
  } else {
    // ------------------------------------------------------------ epilogue --
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const int e = (warp - kEpilogueWarp0) >> 2;  // units e, e + EPI_GROUPS, ... of the CTA
    const uint32_t sbase = smem_u32(out_rows) + (warp - kEpilogueWarp0) * kStageWarpBytes;
    uint32_t acc = e, acc_phase = 0, it_par = 0;
    UnitCursor cur;
    start(cur);
    // Units of this group ahead of the one at hand: the output rows of a unit's
    // columns are loaded two units ahead and their factors, which need the
    // rows, one unit ahead (loads take some 2 us while the SM streams at full
    // rate: with both one unit ahead 8192 tokens' down product took 430 us).
    // Each thread of the group holds the columns tid, tid + 128 and puts them in
    // the group's table when the unit's turn comes (every warp looking all of
    // them up for itself: 326 us).
    const int tid = q * 32 + lane;
    constexpr int PER = (C::TABLE + 127) / 128;
    int* const table = tables + e * (2 * C::TABLE * 2);
    struct Ahead {
      bool has;
      WorkUnit u;
      Item it;
      int valid;
      int orow[PER];
    } now, next;
    float factor[PER];
    auto look_up_rows = [&](Ahead& a, int skip) {
      a.has = true;
      for (; skip >= 0 && a.has; --skip) a.has = cur.next(a.u);
      a.valid = 0;
      int row0 = 0;
      if (a.has) {
        a.it = decode(a.u.item);
        row0 = g_row0[a.it.g] + a.it.n * BN;
        a.valid = min(BN, g_rows[a.it.g] - a.it.n * BN);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = 128 * i + tid;
        a.orow[i] = c >= a.valid ? -1 : args.out_rows != nullptr ? __ldg(args.out_rows + row0 + c) : row0 + c;
      }
    };
    auto look_up_factors = [&](Ahead& a) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (a.orow[i] >= args.n_out) a.orow[i] = -1;
        factor[i] = a.orow[i] >= 0 && args.row_scale != nullptr ? __ldg(args.row_scale + a.orow[i]) : 1.0f;
      }
    };
    look_up_rows(now, e);
    look_up_factors(now);
    look_up_rows(next, C::EPI_GROUPS - 1);
    while (now.has) {
      const Item it = now.it;
      const WorkUnit v = now.u;
      const int valid = now.valid;
      // the table of two units ago: every warp has left it before the barrier below of the unit before
      int* const orow = table + it_par * (2 * C::TABLE);
      float* const factors = reinterpret_cast<float*>(orow + C::TABLE);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = 128 * i + tid;
        if (c < C::TABLE) {
          orow[c] = now.orow[i];
          factors[c] = factor[i];
        }
      }
      now = next;
      look_up_factors(now);
      look_up_rows(next, C::EPI_GROUPS - 1);
      const int feat0 = GATED ? it.m * (kBlockM / 2) + q * 16 : it.m * kBlockM + q * 32;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
      uint64_t* const acc_done = &acc_empty[acc];
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_issuer<PAIR>(acc_done);
      };
      // a part of a split item: if every other part is already stored (the
      // count, read before the wait, says so) this one is the last, and sums
      // the parts straight from tensor memory
      int others_done = 0, fast = 0;
      if (BN <= 32 && v.parts > 1 && q == 0 && lane == 0)
        others_done = ld_acquire_gpu(args.ksplit_cnt + v.slot0) == v.parts - 1;
      // the group's warps take one decision (they meet at this barrier, which
      // the table needs too)
      const bool ok = __all_sync(0xffffffffu, wait_bar<PAIR>(&acc_full[acc], acc_phase, limit, abort_flag));
      volatile int* const oks = s_ok + (e * 2 + it_par) * 4;
      if (lane == 0) oks[q] = ok ? 1 + others_done : 0;
      named_bar_sync(kEpilogueBar + e, 128);
      if (!(oks[0] && oks[1] && oks[2] && oks[3])) {
        if (lane == 0 && !ok) record_abort(abort_flag, args.err);
        break;
      }
      fast = oks[0] == 2;
      it_par ^= 1u;
      tc_fence_after();
      if constexpr (BN <= 32) {
        if (v.parts > 1) {
          const int chunks = (valid + kChunk - 1) / kChunk;
          Chunk c[BN / kChunk];
#pragma unroll
          for (int i = 0; i < BN / kChunk; ++i) {
            if (i >= chunks) break;
            load_chunk(taddr, i * kChunk, c[i]);
            wait_chunk(c[i]);
            if (!fast) store_part<BN>(args.ksplit_part, v.slot, q, i, lane, c[i]);
          }
          release();
          // not the last part so far: stored, counted, and summed by whichever part counts last
          bool last = fast;
          if (!fast) last = ksplit_arrive(args.ksplit_cnt + v.slot0, v.parts, s_last, q == 0 && lane == 0);
          if (last) {
#pragma unroll
            for (int i = 0; i < BN / kChunk; ++i) {
              if (i >= chunks) break;
              sum_parts<BN>(args.ksplit_part, cur, v, fast ? v.part : -1, q, i, lane, c[i]);
              finish_any<GATED>(args, c[i], sbase, orow + i * kChunk, factors + i * kChunk, feat0, lane);
            }
            if (q == 0 && lane == 0) args.ksplit_cnt[v.slot0] = 0;  // ready for the next launch
          }
        } else {
          epilogue_mx<GATED, BN>(args, taddr, feat0, valid, orow, factors, sbase, lane, release);
        }
      } else {
        epilogue_mx<GATED, BN>(args, taddr, feat0, valid, orow, factors, sbase, lane, release);
      }
      acc += C::EPI_GROUPS;
      if (acc >= C::NACC) {
        acc -= C::NACC;
        acc_phase ^= 1u;
      }
    }
  }

  tc_fence_before();
  if constexpr (PAIR) {
    __syncthreads();  // this CTA's roles have ended
    if (threadIdx.x == 0) store_peer(rank ^ 1, peer_abort, *abort_flag);
    __syncwarp();
    cluster_sync();  // neither CTA frees tensor memory or leaves while the other works
    if (*abort_flag || *peer_abort != 0) {  // the same in both
      if (rank == 0 && threadIdx.x == 0) {
        // A stage's fills by the two CTAs differ by one at most (a fill waits for
        // the one before to be read, and it is read when both CTAs have filled it).
        // The even CTA's fill expects the bytes of both.
        constexpr uint32_t kBytes = C::A_BYTES + C::B_BYTES + C::SFA_BYTES;
        for (int s = 0; s < C::STAGES; ++s) {
          const uint64_t mine = fills_of(*own_steps, s, C::STAGES), theirs = fills_of(*peer_steps, s, C::STAGES);
          if (mine > theirs) mbar_complete_tx(&full[s], kBytes);
          if (mine < theirs) mbar_arrive_expect_tx(&full[s], kBytes);
          const uint64_t fills = mine > theirs ? mine : theirs;
          if (fills > 0) mbar_wait(&full[s], static_cast<uint32_t>((fills - 1) & 1), kDrainLimitNs);
        }
      }
      __syncwarp();
      cluster_sync();
    }
  } else {
    __syncthreads();
  }
  pdl_trigger();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else
      tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <bool GATED, int BN>
__global__ void __launch_bounds__(CfgMx<BN>::THREADS, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_s,
                    const __grid_constant__ CUtensorMap map_x, const Mx4GemmArgs args) {
  mx4_gemm_body<GATED, BN>(map_w, map_s, map_x, args);
}
template <bool GATED, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(CfgMx<BN>::THREADS, 1)
    mx4_gemm_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_s,
                         const __grid_constant__ CUtensorMap map_x, const Mx4GemmArgs args) {
  mx4_gemm_body<GATED, BN>(map_w, map_s, map_x, args);
}

__global__ void __launch_bounds__(256)
    tile_scales_kernel(const uint8_t* __restrict__ scales, int N, int gated, int m_stride, int tiles_per_row, int blocks,
                       int scale_ld, uint32_t* __restrict__ tiles, long long n_words) {
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n_words) return;
  // word i: 4 blocks (128 columns) of one row of tile (g, m, k)
  const int in_tile = static_cast<int>(i % (kMx4ScaleTile / 4));
  long long t = i / (kMx4ScaleTile / 4);
  const int k = static_cast<int>(t % tiles_per_row);
  t /= tiles_per_row;
  const int m = static_cast<int>(t % m_stride);
  const long long g = t / m_stride;
  const int r = in_tile / 4 + 32 * (in_tile % 4);
  const int F = N / 2;
  int n = m * kBlockM + r;
  bool have = n < N;
  if (gated) {
    // 16 gate rows, then the up rows of the same features, four times
    const int f = m * (kBlockM / 2) + (r >> 5) * 16 + (r & 15);
    have = f < F;
    n = (r & 16) ? F + f : f;
  }
  uint32_t w = 0;
  if (have) {
    const uint8_t* src = scales + (g * N + n) * scale_ld;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (4 * k + b < blocks) w |= static_cast<uint32_t>(src[4 * k + b]) << (8 * b);
  }
  tiles[i] = w;
}

template <bool GATED, int BN>
auto kernel_of() {
  if constexpr (CfgMx<BN>::PAIR)
    return mx4_gemm_pair_kernel<GATED, BN>;
  else
    return mx4_gemm_kernel<GATED, BN>;
}

template <bool GATED, int BN>
cudaError_t launch_one(const CUtensorMap* map_w, const CUtensorMap* map_s, const CUtensorMap* map_x,
                       const Mx4GemmArgs& a, int num_sms, cudaStream_t stream) {
  return launch_chain(kernel_of<GATED, BN>(), dim3(num_sms / CfgMx<BN>::CTAS * CfgMx<BN>::CTAS),
                      dim3(CfgMx<BN>::THREADS), CfgMx<BN>::SMEM_BYTES, stream, *map_w, *map_s, *map_x, a);
}

template <bool GATED>
cudaError_t dispatch_mx(int tile_n, const CUtensorMap* map_w, const CUtensorMap* map_s, const CUtensorMap* map_x,
                        const Mx4GemmArgs& a, int num_sms, cudaStream_t stream) {
  switch (tile_n) {
    case 16: return launch_one<GATED, 16>(map_w, map_s, map_x, a, num_sms, stream);
    case 32: return launch_one<GATED, 32>(map_w, map_s, map_x, a, num_sms, stream);
    case 64: return launch_one<GATED, 64>(map_w, map_s, map_x, a, num_sms, stream);
    case 96: return launch_one<GATED, 96>(map_w, map_s, map_x, a, num_sms, stream);
    case 128: return launch_one<GATED, 128>(map_w, map_s, map_x, a, num_sms, stream);
    case 240: return launch_one<GATED, 240>(map_w, map_s, map_x, a, num_sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <bool GATED, int BN>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(kernel_of<GATED, BN>(), cudaFuncAttributeMaxDynamicSharedMemorySize,
                              CfgMx<BN>::SMEM_BYTES);
}

template <bool GATED>
cudaError_t prepare_all() {
  cudaError_t e;
  if ((e = prepare_one<GATED, 16>()) != cudaSuccess) return e;
  if ((e = prepare_one<GATED, 32>()) != cudaSuccess) return e;
  if ((e = prepare_one<GATED, 64>()) != cudaSuccess) return e;
  if ((e = prepare_one<GATED, 96>()) != cudaSuccess) return e;
  if ((e = prepare_one<GATED, 128>()) != cudaSuccess) return e;
  return prepare_one<GATED, 240>();
}

}  // namespace

cudaError_t launch_mx4_gemm(bool gated, int tile_n, const CUtensorMap* map_w, const CUtensorMap* map_s,
                            const CUtensorMap* map_x, const Mx4GemmArgs& a, int num_sms, cudaStream_t stream) {
  return gated ? dispatch_mx<true>(tile_n, map_w, map_s, map_x, a, num_sms, stream)
               : dispatch_mx<false>(tile_n, map_w, map_s, map_x, a, num_sms, stream);
}

cudaError_t mx4_gemm_prepare() {
  const cudaError_t e = prepare_all<true>();
  return e != cudaSuccess ? e : prepare_all<false>();
}

cudaError_t launch_mx4_tile_scales(const uint8_t* scales, int G, int N, bool gated, int m_stride, int k_steps,
                                   int blocks, int scale_ld, uint8_t* tiles, cudaStream_t stream) {
  const long long words = static_cast<long long>(G) * m_stride * 2 * k_steps * (kMx4ScaleTile / 4);
  const long long grid = (words + 255) / 256;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  tile_scales_kernel<<<static_cast<unsigned>(grid), 256, 0, stream>>>(
      scales, N, gated, m_stride, 2 * k_steps, blocks, scale_ld, reinterpret_cast<uint32_t*>(tiles), words);
  return cudaGetLastError();
}

}  // namespace moe
