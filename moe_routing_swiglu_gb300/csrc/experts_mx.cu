// MXFP4 SwiGLU experts: the two grouped products of experts_tc.cu on 4-bit
// operands (tcgen05.mma kind::mxf4, block scales of 32 in tensor memory).
//
// Per dispatched row r of expert e, every operand an MXFP4 tensor (E2M1
// elements, one E8M0 scale per 32 of them along K):
//   gate/up  h_r = SiLU(W_gate[e] x_r) * (W_up[e] x_r)    (K = H)
//   down     y_r = W_down[e] h_r                          (K = I)
// The MMA multiplies each element by its scale and accumulates in FP32. h is
// written in the output type, or quantised again to MXFP4 in the epilogue
// (32 channels of a token are one block), or both.
//
// Operand roles as in experts_tc.cu: the MMA's M side (128 TMEM lanes) holds
// weight rows, its N side the expert's tokens, so a decode expert with one
// or two tokens costs N = 16, and two MMAs share each token tile (gate and up
// rows of the same channels, or two blocks of down rows).
//
// A stage is 256 elements of K: one 128-byte swizzle atom per row, four
// MMA steps of 64. Shared memory holds, per stage, two 16 KB weight tiles, the
// token tile, and the scales in the order tcgen05.cp copies to TMEM: atoms of
// 512 bytes, row m of 128 at byte (m % 32) * 16 + (m / 32) * 4, four scale
// bytes (128 elements of K) each. The weights' scales were laid out this way
// once, at the handle's creation (one 1 KB bulk copy per tile and stage);
// the tokens' scales are row-major, because a tile may start at any row, and
// two loader warps place their 32-bit words with cp.async.
//
// One persistent CTA per SM takes tiles blockIdx, blockIdx + grid, ...
//   warp 0 lane 0   producer: TMA of weights, tokens and weight scales
//   warp 1 lane 0   tcgen05.cp of the stage's scales to TMEM, then the MMAs
//                   (both run in issue order); warp 1 also owns the TMEM
//   warps 2..9      epilogue, as in experts_tc.cu
//   warps 10..11    the tokens' scales
// Scales in TMEM have SLOTS buffers; a buffer is rewritten only after the
// MMAs that read it have completed (their stage's "empty" barrier).
//
// Token tiles: an expert's rows are split evenly into ceil(rows / TBN) tiles
// of at most TBN (224: what the 512 TMEM columns hold beside the scales; 32
// for decode, double buffered). Every wait is bounded (about a second), as in
// experts_tc.cu.
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                // weight rows per MMA (TMEM lanes)
constexpr int BK = 256;                // K elements per stage
constexpr int UMMA_K = 64;
constexpr int ROW_BYTES = BK / 2;      // 128 B: one swizzle atom
constexpr int A_BYTES = BM * ROW_BYTES;
constexpr int ATOM = 512;              // scale atom: 128 rows x 4 scale bytes
constexpr int ATOMS_K = BK / 128;      // atoms per 128 rows and stage
constexpr int SFA_BYTES = ATOMS_K * ATOM;
constexpr int NUM_EPI_WARPS = 8;
constexpr int NUM_LOAD_WARPS = 2;
constexpr int FIRST_LOAD_WARP = 2 + NUM_EPI_WARPS;
constexpr int NUM_THREADS = 32 * (2 + NUM_EPI_WARPS + NUM_LOAD_WARPS);
constexpr int XPOSE_BYTES = 2048;      // per-warp transpose buffer: 32 tokens x 32 channels of 16 bits
constexpr int STAGE_SMEM = 200 * 1024; // shared memory given to pipeline stages
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;

template <int TBN>
struct MxCfg {
  static constexpr int GROUPS = (TBN + 127) / 128;           // 128-row groups of the token tile
  static constexpr int B_BYTES = TBN * ROW_BYTES;
  static constexpr int SFB_BYTES = GROUPS * ATOMS_K * ATOM;
  static constexpr int STAGE_BYTES = 2 * A_BYTES + B_BYTES + 2 * SFA_BYTES + SFB_BYTES;
  static constexpr int OFF_B = 2 * A_BYTES;
  static constexpr int OFF_SFA = OFF_B + B_BYTES;
  static constexpr int OFF_SFB = OFF_SFA + 2 * SFA_BYTES;
  static constexpr int STAGES = STAGE_SMEM / STAGE_BYTES;
  // TMEM columns: ACC accumulator buffers of (D0, D1), then SLOTS scale
  // buffers of (SFA0, SFA1, SFB), 4 columns per atom.
  static constexpr int ACC = TBN <= 96 ? 2 : 1;
  static constexpr int SF_COLS = 4 * ATOMS_K * (2 + GROUPS);
  static constexpr int SF_BASE = ACC * 2 * TBN;
  static constexpr int SLOTS_FIT = (512 - SF_BASE) / SF_COLS;
  static constexpr int SLOTS = SLOTS_FIT < STAGES ? SLOTS_FIT : STAGES;
  static constexpr int COLS_USED = SF_BASE + SLOTS * SF_COLS;
  static constexpr uint32_t TMEM_COLS = COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
  static constexpr int SMEM_XPOSE = STAGES * STAGE_BYTES;
  static constexpr int SMEM_BAR = SMEM_XPOSE + NUM_EPI_WARPS * XPOSE_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * ACC + 1;  // full, empty, tfull, tempty, drain
  static constexpr int SMEM_MISC = SMEM_BAR + 8 * NUM_BARS;  // TMEM address, abort flag
  static constexpr int SMEM_TILES = SMEM_MISC + 16;
  static constexpr int SMEM_BYTES = 1024 + SMEM_TILES + 4 * (ROUTE_MAX_E + 1);
  static_assert(STAGE_BYTES % 1024 == 0, "stage alignment");
  static_assert(STAGES >= 3, "pipeline depth");
  static_assert(SLOTS >= 2, "scale buffers");
  static_assert(COLS_USED <= 512, "TMEM columns");
  static_assert(TBN % 32 == 0 && TBN <= 256, "token tile");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// Status codes recorded by a wait that timed out.
constexpr uint32_t ST_PRODUCER_EMPTY = 0x21;
constexpr uint32_t ST_MMA_FULL = 0x22;
constexpr uint32_t ST_MMA_TMEM_EMPTY = 0x23;
constexpr uint32_t ST_EPI_TMEM_FULL = 0x24;
constexpr uint32_t ST_MMA_DRAIN = 0x25;
constexpr uint32_t ST_PRODUCER_DRAIN = 0x26;
constexpr uint32_t ST_LOADER_EMPTY = 0x27;
constexpr uint32_t ST_MMA_SLOT = 0x28;

struct MxArgs {
  const uint32_t* offsets;   // [E + 1]
  const uint8_t* sfa0;       // weight scales in atoms (gate, or down)
  const uint8_t* sfa1;       // up, or down
  const uint8_t* sfb;        // token scales [rows_total, sfb_pitch]
  int sfb_pitch;
  int sf_blocks;             // scale bytes per token row, K / 32
  int row_blocks;            // 128-row blocks of the weight scales per expert
  int E;
  int n_wblocks;             // weight blocks per expert (I/128, or H/256)
  int K;
  int n_out;                 // output columns (I or H)
  uint32_t rows_total;
  uint32_t tile_cap;         // host bound on the tile count
  void* out;                 // [rows_total, n_out] or NULL
  uint8_t* q_codes;          // gate/up: h as MXFP4 [rows_total, n_out / 2] or NULL
  uint8_t* q_scales;         // [rows_total, q_pitch]
  int q_pitch;
  uint32_t* status;
};

// Token tiles of an expert with cnt rows: ceil(cnt / TBN), each of bn rows
// (a multiple of 16) but the last.
template <int TBN>
__device__ __forceinline__ uint32_t token_tiles(uint32_t cnt) { return (cnt + TBN - 1) / TBN; }

struct MxTile {
  int e;
  int w;          // weight block
  uint32_t row0;  // first dispatched row
  int rows;       // valid rows, 1 .. TBN
  int n_tok;      // rows rounded up to 16: the MMA's N
};

template <int TBN>
__device__ __forceinline__ void build_mx_prefix(const uint32_t* __restrict__ offsets, int E, int n_wblocks,
                                                uint32_t* tile_start) {
  const int lane = threadIdx.x & 31;
  uint32_t carry = 0;
  for (int base = 0; base < E; base += 32) {
    const int e = base + lane;
    const uint32_t cnt = e < E ? offsets[e + 1] - offsets[e] : 0u;
    const uint32_t tiles = token_tiles<TBN>(cnt) * static_cast<uint32_t>(n_wblocks);
    uint32_t incl = tiles;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(FULL_MASK, incl, off);
      if (lane >= off) incl += o;
    }
    if (e < E) tile_start[e] = carry + incl - tiles;
    carry += __shfl_sync(FULL_MASK, incl, 31);
  }
  if (lane == 0) tile_start[E] = carry;
}

// Tile -> coordinates; token tiles vary fastest so that the CTAs sharing a
// weight tile run together and read it from L2. Requires tile < tile_start[E].
template <int TBN>
__device__ __forceinline__ MxTile decode_mx_tile(uint32_t tile, const uint32_t* tile_start, int E, int n_wblocks,
                                                 const uint32_t* __restrict__ offsets) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_start[mid] <= tile) lo = mid; else hi = mid;
  }
  MxTile c;
  c.e = lo;
  const uint32_t o0 = offsets[lo];
  const uint32_t cnt = offsets[lo + 1] - o0;
  // The bounds (nt >= 1, bn <= TBN, w < n_wblocks) hold by themselves for
  // valid offsets; for corrupt ones they keep every access in range.
  const uint32_t nt = max(token_tiles<TBN>(cnt), 1u);
  const uint32_t bn = min(((cnt + nt - 1) / nt + 15) & ~15u, static_cast<uint32_t>(TBN));
  const uint32_t local = tile - tile_start[lo];
  const uint32_t w = local / nt;
  const uint32_t m = local - w * nt;
  c.w = static_cast<int>(min(w, static_cast<uint32_t>(n_wblocks - 1)));
  c.row0 = o0 + m * bn;
  const uint32_t done = m * bn;
  const uint32_t left = cnt > done ? cnt - done : 0u;
  c.rows = static_cast<int>(left < bn ? left : bn);
  c.n_tok = c.rows > 0 ? (c.rows + 15) & ~15 : 16;
  return c;
}

// D[tmem] (+)= (A * SFA)[smem] * (B * SFB)[smem]^T, E2M1 elements with one
// E8M0 scale per 32 of K (two per 64-element step, at sfa / sfb in TMEM).
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::mxf4: A and B format E2M1 (bits 7-9 and
// 10-11 = 1), N >> 3 in bits 17-22, scales UE8M0 (bit 23), M >> 7 in bits
// 27-28, and the byte of the 32-bit scale words at which the step's two
// scales start (0 or 2) in bits 4-5 for B and 29-30 for A.
__device__ __forceinline__ uint32_t idesc_mxf4(int N, uint32_t sf_byte) {
  return (sf_byte << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (1u << 27) |
         (sf_byte << 29);
}

// One 512-byte scale atom shared -> TMEM: 32 rows of 16 bytes to 32 lanes x 4
// columns, repeated in all four 32-lane quarters.
__device__ __forceinline__ void tmem_cp_atom(uint32_t taddr, uint32_t smem_addr) {
  // Unswizzled descriptor: 8-row x 16-byte core matrices 128 bytes apart
  // (stride field), version 1.
  const uint64_t d = static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128u >> 4) << 32) |
                     (static_cast<uint64_t>(1u) << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// Untiled bulk copy global -> shared, counted on `bar` (16-byte aligned).
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem_dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// 4-byte global -> shared copy; src_bytes < 4 zero-fills the rest.
__device__ __forceinline__ void cp_async_4(uint32_t dst_smem, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst_smem), "l"(src), "r"(src_bytes) : "memory");
}

// SiLU(g) = g / (1 + e^-g). 16-bit outputs: two approximate functions
// (relative error a few 2^-22, far below the output's rounding); FP32: expf
// and a true division.
template <typename T>
__device__ __forceinline__ float mx_silu(float g) {
  if (std::is_same<T, float>::value) return g / (1.0f + expf(-g));
  return __fdividef(g, 1.0f + __expf(-g));
}

template <typename T, bool GATE_UP, int TBN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    experts_mx_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
                      const __grid_constant__ CUtensorMap tm_b128, const __grid_constant__ CUtensorMap tm_b16,
                      const MxArgs args) {
  using C = MxCfg<TBN>;
  constexpr int STAGES = C::STAGES;
  constexpr int ACC = C::ACC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::SMEM_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;   // [ACC]
  uint64_t* tempty = tfull + ACC;     // [ACC]
  uint64_t* drain = tempty + ACC;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::SMEM_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::SMEM_MISC + 4);
  uint32_t* tile_start = reinterpret_cast<uint32_t*>(smem + C::SMEM_TILES);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1 + 32 * NUM_LOAD_WARPS);  // the producer's expect_tx and each loader thread's copies
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < ACC; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], NUM_EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_a0);
    tma_prefetch_desc(&tm_a1);
    tma_prefetch_desc(&tm_b128);
    tma_prefetch_desc(&tm_b16);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  // From here on the kernel reads what earlier kernels wrote.
  grid_dependency_wait();
  if (warp == 0) build_mx_prefix<TBN>(args.offsets, args.E, args.n_wblocks, tile_start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // The cap keeps a corrupt offsets array from producing an endless tile loop.
  const uint32_t total = min(tile_start[args.E], args.tile_cap);
  const int k_blocks = (args.K + BK - 1) / BK;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0;
      bool ok = true;
      for (uint32_t tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
        const MxTile tc = decode_mx_tile<TBN>(tile, tile_start, args.E, args.n_wblocks, args.offsets);
        const int n128 = tc.n_tok >> 7;
        const int n16 = (tc.n_tok & 127) >> 4;
        const uint32_t tx = static_cast<uint32_t>(2 * A_BYTES + 2 * SFA_BYTES + tc.n_tok * ROW_BYTES);
        const int rb0 = GATE_UP ? tc.w : 2 * tc.w;
        const int rb1 = GATE_UP ? tc.w : 2 * tc.w + 1;
        const int64_t sf_expert = static_cast<int64_t>(tc.e) * args.row_blocks;
        const uint8_t* s0 = args.sfa0 + (sf_expert + rb0) * k_blocks * SFA_BYTES;
        const uint8_t* s1 = args.sfa1 + (sf_expert + rb1) * k_blocks * SFA_BYTES;
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, args.status, ST_PRODUCER_EMPTY,
                                 WAIT_LIMIT_NS)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + stage * C::STAGE_BYTES;
          const int k0 = kb * ROW_BYTES;
          mbar_arrive_expect_tx(&full[stage], tx);
          tma_load_3d(st, &tm_a0, &full[stage], k0, rb0 * BM, tc.e);
          tma_load_3d(st + A_BYTES, &tm_a1, &full[stage], k0, rb1 * BM, tc.e);
          bulk_load(st + C::OFF_SFA, s0 + static_cast<int64_t>(kb) * SFA_BYTES, SFA_BYTES, &full[stage]);
          bulk_load(st + C::OFF_SFA + SFA_BYTES, s1 + static_cast<int64_t>(kb) * SFA_BYTES, SFA_BYTES, &full[stage]);
          uint8_t* b_dst = st + C::OFF_B;
          int r = 0;
          for (int b = 0; b < n128; ++b, r += 128)
            tma_load_2d(b_dst + r * ROW_BYTES, &tm_b128, &full[stage], k0, static_cast<int>(tc.row0) + r);
          for (int b = 0; b < n16; ++b, r += 16)
            tma_load_2d(b_dst + r * ROW_BYTES, &tm_b16, &full[stage], k0, static_cast<int>(tc.row0) + r);
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      launch_dependents();  // this CTA issues no more loads
      if (!ok) {
        // Let the copies already in flight land before the block can exit.
        const uint32_t n_back = issued < STAGES ? issued : STAGES;
        for (uint32_t i = 1; i <= n_back; ++i) {
          const uint32_t n = issued - i;
          mbar_wait_bounded(&full[n % STAGES], (n / STAGES) & 1u, nullptr, args.status, ST_PRODUCER_DRAIN,
                            WAIT_LIMIT_NS);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ scales to TMEM, MMAs
    if (lane == 0) {
      uint32_t n = 0;  // stages consumed
      bool ok = true;
      uint32_t it = 0;
      for (uint32_t tile = blockIdx.x; ok && tile < total; tile += gridDim.x, ++it) {
        const MxTile tc = decode_mx_tile<TBN>(tile, tile_start, args.E, args.n_wblocks, args.offsets);
        const uint32_t idesc0 = idesc_mxf4(tc.n_tok, 0), idesc2 = idesc_mxf4(tc.n_tok, 2);
        const int groups = (tc.n_tok + 127) >> 7;
        const uint32_t acc = it % ACC;
        if (!mbar_wait_bounded(&tempty[acc], ((it / ACC) & 1u) ^ 1u, abort_flag, args.status, ST_MMA_TMEM_EMPTY,
                               WAIT_LIMIT_NS)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d0 = tmem_base + acc * (2 * TBN);
        for (int kb = 0; kb < k_blocks; ++kb, ++n) {
          const uint32_t stage = n % STAGES;
          if (!mbar_wait_bounded(&full[stage], (n / STAGES) & 1u, abort_flag, args.status, ST_MMA_FULL,
                                 WAIT_LIMIT_NS)) {
            ok = false;
            break;
          }
          if (C::SLOTS < STAGES && n >= static_cast<uint32_t>(C::SLOTS)) {
            // The scale buffer's previous readers: the MMAs of stage n - SLOTS.
            const uint32_t p = n - C::SLOTS;
            if (!mbar_wait_bounded(&empty[p % STAGES], (p / STAGES) & 1u, abort_flag, args.status, ST_MMA_SLOT,
                                   WAIT_LIMIT_NS)) {
              ok = false;
              break;
            }
          }
          fence_proxy_async_smem();  // the loaders' cp.async (generic proxy) before tcgen05.cp
          tc_fence_after();
          const uint32_t st = smem_u32(smem + stage * C::STAGE_BYTES);
          const uint32_t sf = tmem_base + C::SF_BASE + (n % C::SLOTS) * C::SF_COLS;
          const uint32_t sfb = sf + 8 * ATOMS_K;
#pragma unroll
          for (int a = 0; a < ATOMS_K; ++a) {
            tmem_cp_atom(sf + 4 * a, st + C::OFF_SFA + a * ATOM);
            tmem_cp_atom(sf + 4 * ATOMS_K + 4 * a, st + C::OFF_SFA + SFA_BYTES + a * ATOM);
            for (int g = 0; g < groups; ++g)
              tmem_cp_atom(sfb + 4 * (a * C::GROUPS + g), st + C::OFF_SFB + (a * C::GROUPS + g) * ATOM);
          }
          const int left = args.K - kb * BK;  // MMA steps wholly past K are left out
          const uint32_t a0 = st, a1 = st + A_BYTES, b = st + C::OFF_B;
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k) {
            if (k * UMMA_K < left) {
              const uint32_t accum = (kb > 0 || k > 0) ? 1u : 0u;
              const uint32_t id = (k & 1) != 0 ? idesc2 : idesc0;
              const uint64_t bd = sdesc_kmajor_sw128(b + k * (UMMA_K / 2));
              const uint32_t sb = sfb + 4 * (k >> 1) * C::GROUPS;
              umma_mxf4(d0, sdesc_kmajor_sw128(a0 + k * (UMMA_K / 2)), bd, id, sf + 4 * (k >> 1), sb, accum);
              umma_mxf4(d0 + TBN, sdesc_kmajor_sw128(a1 + k * (UMMA_K / 2)), bd, id,
                        sf + 4 * ATOMS_K + 4 * (k >> 1), sb, accum);
            }
          }
          umma_commit(&empty[stage]);
        }
        if (!ok) break;
        umma_commit(&tfull[acc]);
      }
      // Every copy and MMA issued above completes before TMEM is released.
      umma_commit(drain);
      mbar_wait_bounded(drain, 0, nullptr, args.status, ST_MMA_DRAIN, WAIT_LIMIT_NS);
    }
    __syncwarp();
  } else if (warp < FIRST_LOAD_WARP) {
    // ------------------------------------------------------------ epilogue
    constexpr int TOK = XPOSE_BYTES / (32 * static_cast<int>(sizeof(T)));  // tokens per transpose: 32, or 16 for FP32
    const int ew = warp - 2;
    const int quad = warp & 3;                  // TMEM lanes 32*quad ..
    const int half = ew >> 2;                   // takes 32-token chunks half, half+2, ...
    uint8_t* xp = smem + C::SMEM_XPOSE + ew * XPOSE_BYTES;
    T* xt = reinterpret_cast<T*>(xp);
    uint32_t it = 0;
    for (uint32_t tile = blockIdx.x; tile < total; tile += gridDim.x, ++it) {
      const MxTile tc = decode_mx_tile<TBN>(tile, tile_start, args.E, args.n_wblocks, args.offsets);
      const uint32_t acc = it % ACC;
      const bool ok = mbar_wait_bounded(&tfull[acc], (it / ACC) & 1u, abort_flag, args.status, ST_EPI_TMEM_FULL,
                                        WAIT_LIMIT_NS);
      if (!__all_sync(FULL_MASK, ok)) break;  // tcgen05.ld is warp-collective: the whole warp goes on or stops
      tc_fence_after();
      const uint32_t t_lane = tmem_base + acc * (2 * TBN) + (static_cast<uint32_t>(quad * 32) << 16);
      const int64_t colA = static_cast<int64_t>(tc.w) * (GATE_UP ? BM : 2 * BM) + quad * 32;
      for (int c0 = 32 * half; c0 < tc.n_tok; c0 += 64) {
        uint32_t v0[32], v1[32];
        tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(c0), v0);
        tmem_ld_32x32b_x32(t_lane + TBN + static_cast<uint32_t>(c0), v1);
        tmem_ld_wait();
#pragma unroll
        for (int blk = 0; blk < (GATE_UP ? 1 : 2); ++blk) {
          const int64_t col0 = colA + blk * BM;
          const bool col_ok = col0 < args.n_out;  // n_out is a multiple of 32: the warp's block is in or out
#pragma unroll
          for (int t0 = 0; t0 < 32; t0 += TOK) {
            // Lane = output channel, register = token: write token rows.
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
              float val;
              if (GATE_UP) val = mx_silu<T>(__uint_as_float(v0[t0 + j])) * __uint_as_float(v1[t0 + j]);
              else val = __uint_as_float(blk == 0 ? v0[t0 + j] : v1[t0 + j]);
              xt[j * 32 + lane] = from_f32<T>(val);
            }
            __syncwarp();
            if (args.out != nullptr) {
              constexpr int PARTS = 32 * static_cast<int>(sizeof(T)) / 16;  // 16-byte runs per token row
              constexpr int TPP = 32 / PARTS;                               // tokens per pass
              const int part = lane % PARTS;
#pragma unroll
              for (int p = 0; p < TOK / TPP; ++p) {
                const int j = p * TPP + lane / PARTS;
                const uint4 row = *reinterpret_cast<const uint4*>(xp + (j * PARTS + part) * 16);
                const int t_in = c0 + t0 + j;
                if (t_in < tc.rows && tc.row0 + static_cast<uint32_t>(t_in) < args.rows_total && col_ok) {
                  T* dst = static_cast<T*>(args.out) + (static_cast<int64_t>(tc.row0) + t_in) * args.n_out + col0;
                  reinterpret_cast<uint4*>(dst)[part] = row;
                }
              }
            }
            if (GATE_UP && args.q_codes != nullptr) {
              // One lane per token: its 32 channels are one block. The
              // 16-byte runs are read in a lane-rotated order so that a
              // quarter-warp's reads fall into different banks.
              const int j = lane % TOK;
              float v[32];
              uint32_t amax = 0;
              constexpr int RUNS = 32 * static_cast<int>(sizeof(T)) / 16;
              constexpr int EPR = 16 / static_cast<int>(sizeof(T));
#pragma unroll
              for (int q = 0; q < RUNS; ++q) {
                const int run = sizeof(T) == 2 ? ((q + (j >> 1)) & (RUNS - 1)) : ((q + j) & (RUNS - 1));
                const uint4 raw = *reinterpret_cast<const uint4*>(xp + (j * RUNS + run) * 16);
                const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
                for (int i = 0; i < EPR; ++i) {
                  v[q * EPR + i] = to_f32(e[i]);
                  amax = max(amax, __float_as_uint(v[q * EPR + i]) & 0x7FFFFFFFu);
                }
              }
              const uint32_t byte = mx_scale_byte(amax);
              const float s = mx_inv_scale(byte);
              uint32_t w[4];
              // v[8q ..] holds elements 8 ((q + rot) % 4) .. of the token
              // (FP32: runs of 4, rotated by an even or odd number of them).
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float e8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) e8[i] = v[q * 8 + i] * s;
                w[q] = byte == 255u ? 0u : mx_pack8(e8);
              }
              uint32_t o[4];
              if (sizeof(T) == 2) {
                const int rot = (j >> 1) & 3;
#pragma unroll
                for (int d = 0; d < 4; ++d) {  // word d was read at step (d - rot) % 4
                  const int q = (d - rot) & 3;
                  o[d] = q == 0 ? w[0] : q == 1 ? w[1] : q == 2 ? w[2] : w[3];
                }
              } else {
                // 16-bit halves: half h (4 elements) was read at step (h - j) % 8.
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                  uint32_t lo = 0, hi = 0;
#pragma unroll
                  for (int q = 0; q < 8; ++q) {
                    const uint32_t hw = (w[q >> 1] >> (16 * (q & 1))) & 0xFFFFu;
                    if (q == ((2 * d - j) & 7)) lo = hw;
                    if (q == ((2 * d + 1 - j) & 7)) hi = hw;
                  }
                  o[d] = lo | (hi << 16);
                }
              }
              const int t_in = c0 + t0 + j;
              if (lane < TOK && t_in < tc.rows && tc.row0 + static_cast<uint32_t>(t_in) < args.rows_total && col_ok) {
                const int64_t r = static_cast<int64_t>(tc.row0) + t_in;
                *reinterpret_cast<uint4*>(args.q_codes + r * (args.n_out / 2) + col0 / 2) =
                    make_uint4(o[0], o[1], o[2], o[3]);
                uint8_t* sp = args.q_scales + r * args.q_pitch;
                sp[col0 / MX_BLOCK] = static_cast<uint8_t>(byte);
                if (col0 + MX_BLOCK >= args.n_out)
                  for (int p = static_cast<int>(col0 / MX_BLOCK) + 1; p < args.q_pitch; ++p) sp[p] = 0;
              }
            }
            __syncwarp();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
    }
  } else {
    // ------------------------------------------------------------ the tokens' scales
    // Word a of token n (its four scale bytes for K elements 256 kb + 128 a
    // ..) goes to atom (a, n / 128). Bytes past K / 32 and rows past the tile
    // are filled with 0, never read.
    const int lt = threadIdx.x - 32 * FIRST_LOAD_WARP;   // 0 .. 63
    uint32_t n = 0;
    for (uint32_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const MxTile tc = decode_mx_tile<TBN>(tile, tile_start, args.E, args.n_wblocks, args.offsets);
      bool ok = true;
      for (int kb = 0; kb < k_blocks; ++kb, ++n) {
        const uint32_t stage = n % STAGES;
        ok = mbar_wait_bounded(&empty[stage], ((n / STAGES) & 1u) ^ 1u, abort_flag, args.status, ST_LOADER_EMPTY,
                               WAIT_LIMIT_NS);
        if (!__all_sync(FULL_MASK, ok)) {
          ok = false;
          break;
        }
        const uint32_t sfb = smem_u32(smem + stage * C::STAGE_BYTES + C::OFF_SFB);
        for (int i = lt; i < tc.n_tok * ATOMS_K; i += 32 * NUM_LOAD_WARPS) {
          const int tok = i / ATOMS_K, a = i % ATOMS_K;
          const uint32_t dst = sfb + static_cast<uint32_t>((a * C::GROUPS + (tok >> 7)) * ATOM + (tok & 31) * 16 +
                                                           ((tok >> 5) & 3) * 4);
          const int byte0 = (kb * ATOMS_K + a) * 4;
          int valid = args.sf_blocks - byte0;
          valid = valid < 0 ? 0 : valid > 4 ? 4 : valid;
          const uint32_t row = tc.row0 + static_cast<uint32_t>(tok);
          if (tok >= tc.rows || row >= args.rows_total) valid = 0;
          const uint8_t* src = valid > 0 ? args.sfb + static_cast<int64_t>(row) * args.sfb_pitch + byte0 : args.sfb;
          cp_async_4(dst, src, static_cast<uint32_t>(valid));
        }
        cp_async_mbar_arrive_noinc(&full[stage]);
      }
      if (!ok) break;
    }
    cp_async_wait_all();  // no copy may land after the block has exited
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn_mx() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
  });
  return fn;
}

// [E, rows, row_bytes] codes, box 128 bytes x box_rows x 1.
bool encode_codes(CUtensorMap* m, const void* ptr, uint64_t row_bytes, uint64_t rows, uint64_t E, uint32_t box_rows,
                  int rank) {
  auto fn = encode_fn_mx();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {row_bytes, rows, E};
  const cuuint64_t strides[2] = {row_bytes, rows * row_bytes};
  const cuuint32_t box[3] = {ROW_BYTES, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank), const_cast<void*>(ptr), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool GATE_UP, int TBN>
cudaError_t launch_mx(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b128, const CUtensorMap& b16,
                      MxArgs args, int64_t rows, int num_sms, cudaStream_t stream) {
  auto kern = experts_mx_kernel<T, GATE_UP, TBN>;
  constexpr int SMEM_BYTES = MxCfg<TBN>::SMEM_BYTES;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (err != cudaSuccess) return err;
  // At most ceil(rows_e / TBN) token tiles per expert.
  const int64_t cap = (rows / TBN + (rows < args.E ? rows : args.E)) * args.n_wblocks;
  args.tile_cap = static_cast<uint32_t>(cap < 0xFFFFFFFFll ? cap : 0xFFFFFFFFll);
  const int grid = static_cast<int>(cap < num_sms ? cap : num_sms);
  return launch_dependent(kern, dim3(grid), dim3(NUM_THREADS), SMEM_BYTES, stream, a0, a1, b128, b16, args);
}

template <typename T>
cudaError_t stage_t(const MxWeights& w, bool gate_up, const CUtensorMap& b128, const CUtensorMap& b16,
                    const MxArgs& args, int64_t rows, int num_sms, cudaStream_t stream) {
  // Decode-sized batches (at most 8 rows per expert on average) take
  // 32-token tiles: more weight bytes in flight and double-buffered
  // accumulators; larger ones 224-token tiles, which read each weight tile
  // for seven times the tokens.
  const bool small = rows <= 8 * static_cast<int64_t>(args.E);
  if (gate_up)
    return small ? launch_mx<T, true, 32>(w.gate, w.up, b128, b16, args, rows, num_sms, stream)
                 : launch_mx<T, true, 224>(w.gate, w.up, b128, b16, args, rows, num_sms, stream);
  return small ? launch_mx<T, false, 32>(w.down, w.down, b128, b16, args, rows, num_sms, stream)
               : launch_mx<T, false, 224>(w.down, w.down, b128, b16, args, rows, num_sms, stream);
}

}  // namespace

int64_t mx_weight_row_blocks(bool gate_up, int64_t R) {
  return gate_up ? (R + BM - 1) / BM : (R + 2 * BM - 1) / (2 * BM) * 2;
}

size_t mx_weight_scale_bytes(bool gate_up, int64_t E, int64_t R, int64_t K) {
  return static_cast<size_t>(E) * static_cast<size_t>(mx_weight_row_blocks(gate_up, R)) *
         static_cast<size_t>((K + BK - 1) / BK) * SFA_BYTES;
}

bool mx_encode_weights(const void* gate, const void* up, const void* down, int64_t E, int64_t H, int64_t I,
                       MxWeights* out, const char** why) {
  if (encode_fn_mx() == nullptr) {
    *why = "the CUDA driver does not provide cuTensorMapEncodeTiled";
    return false;
  }
  if (!encode_codes(&out->gate, gate, H / 2, I, E, BM, 3) || !encode_codes(&out->up, up, H / 2, I, E, BM, 3) ||
      !encode_codes(&out->down, down, I / 2, H, E, BM, 3)) {
    *why = "cuTensorMapEncodeTiled rejected an expert weight tensor map";
    return false;
  }
  return true;
}

cudaError_t launch_experts_mx(const MxWeights& w, bool gate_up, const void* codes, const void* scales,
                              const uint32_t* offsets, int E, int64_t rows, int64_t H, int64_t I, moe_dtype out_dtype,
                              void* out, void* q_codes, void* q_scales, int num_sms, cudaStream_t stream,
                              const char** why) {
  if (rows == 0) return cudaSuccess;
  const int64_t K = gate_up ? H : I;
  const int64_t N = gate_up ? I : H;
  CUtensorMap b128, b16;
  if (!encode_codes(&b128, codes, K / 2, rows, 1, 128, 2) || !encode_codes(&b16, codes, K / 2, rows, 1, 16, 2)) {
    *why = "cuTensorMapEncodeTiled rejected the token tensor map";
    return cudaErrorInvalidValue;
  }
  MxArgs a{};
  cudaError_t err = device_status_ptr(&a.status);
  if (err != cudaSuccess) return err;
  a.offsets = offsets;
  a.sfa0 = static_cast<const uint8_t*>(gate_up ? w.gate_sf : w.down_sf);
  a.sfa1 = static_cast<const uint8_t*>(gate_up ? w.up_sf : w.down_sf);
  a.sfb = static_cast<const uint8_t*>(scales);
  a.sfb_pitch = static_cast<int>(mx_scale_pitch(K));
  a.sf_blocks = static_cast<int>(K / MX_BLOCK);
  a.row_blocks = static_cast<int>(mx_weight_row_blocks(gate_up, N));
  a.E = E;
  a.n_wblocks = static_cast<int>(gate_up ? (N + BM - 1) / BM : (N + 2 * BM - 1) / (2 * BM));
  a.K = static_cast<int>(K);
  a.n_out = static_cast<int>(N);
  a.rows_total = static_cast<uint32_t>(rows);
  a.out = out;
  a.q_codes = static_cast<uint8_t*>(q_codes);
  a.q_scales = static_cast<uint8_t*>(q_scales);
  a.q_pitch = static_cast<int>(mx_scale_pitch(N));
  if (out_dtype == MOE_F32) return stage_t<float>(w, gate_up, b128, b16, a, rows, num_sms, stream);
  if (out_dtype == MOE_F16) return stage_t<__half>(w, gate_up, b128, b16, a, rows, num_sms, stream);
  return stage_t<__nv_bfloat16>(w, gate_up, b128, b16, a, rows, num_sms, stream);
}

}  // namespace moe
