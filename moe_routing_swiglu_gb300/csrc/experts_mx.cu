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
// weight rows, its N side the expert's tokens (16 at least: what an MMA of
// N = 16 takes was not measured apart, decode is bound by the weights' bytes),
// and two MMAs share each token tile (gate and up rows of the same channels,
// or two blocks of down rows).
//
// A stage is 256 elements of K: one 128-byte swizzle atom per row, four MMA
// steps of 64; shared memory holds STAGES of two 16 KB weight tiles and the
// token tile. Scales travel apart, in a deeper ring: the MMA reads them from
// TMEM as atoms of 128 rows x 4 bytes (128 elements of K), row m in lane
// m % 32, column m / 32, repeated in the four 32-lane quarters. The weights'
// scales were laid out as such atoms once, at the handle's creation (one 2 KB
// bulk copy per stage); the tokens' scales are row-major, because a tile may
// start at any row, and are placed word by word with cp.async.
//
// One persistent CTA per SM takes tiles blockIdx, blockIdx + grid, ... (the
// five roles find their tiles alone: no counter to clear before the launch and
// no ring of claimed tiles between them; the price is a last round as long as
// its longest tile, which counts where there are few rounds: 504 tiles in the
// decode step of 84 touched experts at I=768. Claiming was not tried here).
//   warp 0 lane 0   producer: TMA of weights and tokens
//   warp 1 lane 0   MMAs; warp 1 also owns the TMEM
//   warps 2..17     epilogue: accumulators to registers in fragment order,
//                   packed in token pairs, transposed by stmatrix into token
//                   rows, which leave by bulk tensor stores (or quantised)
//   warps 18..21    scales, shared -> TMEM by tcgen05.st into one of SLOTS
//                   buffers, rewritten only after the MMAs that read it
//   warp 22         scales, global -> shared
// The scales go to TMEM by stores and not by tcgen05.cp because the copies
// run on the tensor pipe in turn with the MMAs: eight a stage took 0.2 to
// 0.3 us beside 0.5 us of MMAs.
//
// What bounds it (gate/up of 16384 rows, E=8, H=4096, I=14336: 640-650 us in
// repeated calls on the same operands, 5.9-6.0 PFLOP/s; 685-700 us when every
// call gets new ones): an MMA takes about 128 clocks at N = 112 as at N = 208
// (from a stage's time without loads and epilogue), 8 a stage, 467 us in all;
// the loads bring 63.5 KB a stage into each SM, 48 bytes a clock and SM on
// average (profile of 4096 rows: 1.32 GB from L2 in 105 us), and take nearly as
// long; the pipeline without the epilogue takes 537 us, and the epilogue's
// reads of the accumulators are overlapped by nothing but the loads of the next
// tile's first stages: two accumulators would need 832 TMEM columns. Tried and
// slower: N <= 112 with two accumulators (twice the MMAs; 1061 us when N <= 208
// took 712), one weight tile per MMA with two accumulators (half the work a
// stage for the same 0.25 us of waits; 979 us when two took 680).
//
// Token tiles: an expert's rows are split evenly into ceil(rows / 208) tiles of
// at most 208 tokens, what the 512 TMEM columns hold beside three scale
// buffers. Decode batches take the same tiles: 32-token ones with more stages
// and two accumulators measured within 6 % of them, either way, at 1 to 24
// rows per expert (gate/up in us, 32 / 208 tokens: 30.6 / 30.6 at one row and
// 41.7 / 42.9 at 24 for E=128, H=2048, I=768; 81.6 / 79.6 at 24 for E=8,
// H=4096, I=14336, whose down products they ran in 44.0 / 46.3), and behind
// from 32 rows on (45.1 / 42.5, 96.6 / 79.8). Every wait is bounded (about
// a second), as in experts_tc.cu.
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "moe_common.cuh"
#include "moe_internal.h"
#include "mxfp4.cuh"
#include "ring_drain.h"

namespace moe {
namespace {

constexpr int BM = 128;                // weight rows per MMA (TMEM lanes)
constexpr int BK = 256;                // K elements per stage
constexpr int UMMA_K = 64;
constexpr int ROW_BYTES = BK / 2;      // 128 B: one swizzle atom
constexpr int A_BYTES = BM * ROW_BYTES;
constexpr int ATOM = 512;              // scale atom: 128 rows x 4 scale bytes
constexpr int ATOMS_K = BK / 128;      // atoms per 128 rows and stage
constexpr int SFA_BYTES = 2 * ATOMS_K * ATOM;  // scales of both weight tiles of a stage
constexpr int NUM_EPI_WARPS = 16;     // four per 32 TMEM lanes
constexpr int FIRST_SCALE_WARP = 2 + NUM_EPI_WARPS;  // four warps, one per 32 TMEM lanes
constexpr int LOAD_WARP = FIRST_SCALE_WARP + 4;
constexpr int NUM_THREADS = 32 * (LOAD_WARP + 1);
constexpr int EPI_TOKENS = 16;         // tokens an epilogue warp takes at a time
constexpr int XPOSE_BYTES = 1024;      // its transpose buffer: 16 tokens x 32 channels of 16 bits
constexpr int TBN = 208;               // most tokens of a tile: the MMA's N
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;

struct MxCfg {
  static constexpr int GROUPS = (TBN + 127) / 128;           // 128-row groups of the token tile
  static constexpr int STAGE_BYTES = 2 * A_BYTES + TBN * ROW_BYTES;
  static constexpr int OFF_B = 2 * A_BYTES;
  static constexpr int STAGES = 184 * 1024 / STAGE_BYTES;
  static constexpr int SFB_BYTES = GROUPS * ATOMS_K * ATOM;
  static constexpr int SF_BYTES = SFA_BYTES + SFB_BYTES;     // a stage's scales: their own, deeper ring
  static constexpr int SF_STAGES = 6;
  // TMEM columns: the accumulators D0 and D1, then SLOTS scale buffers of
  // (SFA0, SFA1, SFB), 4 columns per atom.
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int SF_COLS = 4 * ATOMS_K * (2 + GROUPS);
  static constexpr int SF_BASE = 2 * TBN;
  static constexpr int SLOTS = (static_cast<int>(TMEM_COLS) - SF_BASE) / SF_COLS;
  static constexpr int SMEM_SF = STAGES * STAGE_BYTES;
  static constexpr int SMEM_XPOSE = SMEM_SF + SF_STAGES * SF_BYTES;
  static constexpr int SMEM_BAR = SMEM_XPOSE + NUM_EPI_WARPS * XPOSE_BYTES;
  // full, empty; sf_full, sf_empty; sf_ready; tfull, tempty; drain
  static constexpr int NUM_BARS = 2 * STAGES + 2 * SF_STAGES + SLOTS + 3;
  static constexpr int SMEM_MISC = SMEM_BAR + 8 * NUM_BARS;  // TMEM address, abort flag, stages issued by the two loaders
  static constexpr int SMEM_TILES = SMEM_MISC + 16;          // tile prefix, then the row offsets
  static constexpr int SMEM_BYTES = 1024 + SMEM_TILES + 8 * (ROUTE_MAX_E + 1);
  static_assert(STAGE_BYTES % 1024 == 0, "swizzle atom alignment");
  static_assert(STAGES >= 3, "pipeline depth");
  // Every role walks the stages one by one, so each of its waits by parity
  // follows on the one before; and a stage's barrier cannot advance twice
  // before the scale warps have looked at it, because its next MMAs need scales
  // that they write after.
  static_assert(SLOTS >= 2 && SLOTS <= STAGES, "scale buffers");
  static_assert(SF_COLS % 8 == 0, "scale stores of 8 columns");
  static_assert(TBN % 16 == 0 && TBN <= 256, "token tile");
  static_assert(SMEM_XPOSE % 512 == 0, "the transpose buffers start on the 64-byte swizzle's period");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// Status codes recorded by a wait that timed out.
constexpr uint32_t ST_PRODUCER_EMPTY = 0x31;
constexpr uint32_t ST_MMA_FULL = 0x32;
constexpr uint32_t ST_MMA_TMEM_EMPTY = 0x33;
constexpr uint32_t ST_EPI_TMEM_FULL = 0x34;
constexpr uint32_t ST_MMA_DRAIN = 0x35;
constexpr uint32_t ST_PRODUCER_DRAIN = 0x36;
constexpr uint32_t ST_LOADER_EMPTY = 0x37;
constexpr uint32_t ST_SCALE_SLOT = 0x38;
constexpr uint32_t ST_SCALE_FULL = 0x39;
constexpr uint32_t ST_MMA_SF_READY = 0x3A;
constexpr uint32_t ST_LOADER_DRAIN = 0x3B;

struct MxArgs {
  const uint32_t* offsets;   // [E + 1]
  const uint8_t* sfa;        // weight scales in atoms, [E, n_wblocks, K / 128, 2, ATOM]
  const uint8_t* sfb;        // token scales [rows_total, sfb_pitch]
  int sfb_pitch;
  int sf_blocks;             // scale bytes per token row, K / 32
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

// Token rows come in boxes of 128, 64, 32 and 16 rows, the binary digits of
// the tile's N: at most four copies a stage.
constexpr int NUM_BOXES = 4;
struct MxMaps {
  CUtensorMap a0;            // gate, or down (256-row box)
  CUtensorMap a1;            // up
  CUtensorMap b[NUM_BOXES];
  CUtensorMap out;           // 16-bit outputs: boxes of 32 columns x 16 rows, 64-byte swizzle
};

// Token tiles of an expert with cnt rows: ceil(cnt / TBN), each of bn rows
// (a multiple of 16) but the last.
__device__ __forceinline__ uint32_t token_tiles(uint32_t cnt) { return (cnt + TBN - 1) / TBN; }

struct MxTile {
  int e;
  int w;          // weight block
  uint32_t row0;  // first dispatched row
  int rows;       // valid rows, 1 .. TBN
  int n_tok;      // rows rounded up to 16: the MMA's N
};

// Exclusive prefix of the experts' tiles, tile_start[0..E], and a copy of the
// offsets, by one warp. Eight experts' counts per lane are loaded before they
// are used: one trip to memory for 256 experts. Offsets past
// the buffers' rows count as the end of the buffers.
__device__ __forceinline__ void build_mx_prefix(const uint32_t* __restrict__ offsets, int E, uint32_t rows_total,
                                                int n_wblocks, uint32_t* tile_start, uint32_t* offs) {
  constexpr int BATCH = 8;
  const int lane = threadIdx.x & 31;
  uint32_t carry = 0;
  for (int base = 0; base < E; base += 32 * BATCH) {
    uint32_t lo[BATCH], hi[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int e = base + 32 * i + lane;
      lo[i] = e < E ? min(offsets[e], rows_total) : 0u;
      hi[i] = e < E ? max(min(offsets[e + 1], rows_total), lo[i]) : 0u;
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int e = base + 32 * i + lane;
      if (base + 32 * i >= E) break;
      const uint32_t tiles = token_tiles(hi[i] - lo[i]) * static_cast<uint32_t>(n_wblocks);
      uint32_t incl = tiles;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(FULL_MASK, incl, off);
        if (lane >= off) incl += o;
      }
      if (e < E) {
        tile_start[e] = carry + incl - tiles;
        offs[e] = lo[i];
        if (e == E - 1) offs[E] = hi[i];
      }
      carry += __shfl_sync(FULL_MASK, incl, 31);
    }
  }
  if (lane == 0) tile_start[E] = carry;
}

// Tile -> coordinates; token tiles vary fastest so that the CTAs sharing a
// weight tile run together and read it from L2. Requires tile < tile_start[E].
__device__ __forceinline__ MxTile decode_mx_tile(uint32_t tile, const uint32_t* tile_start, int E, int n_wblocks,
                                                 const uint32_t* offsets) {
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
  const uint32_t nt = max(token_tiles(cnt), 1u);
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

// Eight TMEM columns of this warp's 32 lanes (lane i of the warp writes TMEM
// lane base + i).
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, uint4 a, uint4 b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Tensor store shared -> global of one box of a 2-D map, in the issuing
// thread's current bulk async-group.
__device__ __forceinline__ void tma_store_2d(const void* desc, uint32_t smem_src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(desc), "r"(c0),
               "r"(c1), "r"(smem_src)
               : "memory");
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

// SiLU(g) = g / (1 + e^-g) as 2^-8 g times the hardware's reciprocal of
// 2^-8 (1 + e^-g). Without the 2^-8, e^-g overflows (or its reciprocal is
// flushed) from g = -87 down, while the SiLU is a normal number of FP32 (and
// BF16) to g = -92, and u may bring it back to any size. With it the power and
// the reciprocal leave FP32 only where the SiLU is below 2^-126; there it may
// count as 0.
//
// 16-bit outputs: the hardware's 2^x. Relative error a few 2^-22 and |g| 2^-23,
// below 2^-16: far under the output's rounding. FP32: e^-g as the square of
// expf(-g / 2), whose 2 ulp count twice: with the reciprocal's ulp and two
// roundings less than 2^-20, under what the sum of K >= 32 products may be off
// by. (With a true division in its place the FP32 product of 16384 rows, E=8,
// H=4096, I=14336 takes 924 us instead of 756; the 16-bit one 642 either way.)
template <typename T>
__device__ __forceinline__ float mx_silu(float g) {
  float d, r;
  if (std::is_same<T, float>::value) {
    const float h = expf(-0.5f * g);
    d = fmaf(h * 0x1p-8f, h, 0x1p-8f);
  } else {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(-1.4426950408889634f, g, -8.0f)));
    d = e + 0x1p-8f;
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return (g * 0x1p-8f) * r;
}

// 16 columns of 16 TMEM lanes, in the order of a matrix fragment: thread t
// gets, for each group i of 8 columns, columns 8i + 2 (t % 4) and the next of
// lane t / 4 (r[4i], r[4i + 1]) and of lane t / 4 + 8 (r[4i + 2], r[4i + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// 16 columns of this warp's 32 TMEM lanes (one lane a thread).
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Four 8 x 8 matrices of 16-bit elements from fragments, each transposed:
// element [row t / 4][2 (t % 4) ..] of matrix q goes to the 16-byte row that
// lane 8 q + column addresses.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// A warp's tokens x 32 channels in shared memory, one block of 32 per token,
// quantised: LPT lanes share a token, each with two 16-byte runs (run(tok, q):
// the address of the token's run q). The values come rounded to T, also where h
// itself is not stored: a call that fuses the quantisation gives the bytes that
// h and moe_mxfp4_quantize give (an F16 h beyond 65504 is an infinity in both,
// and its block NaN). Row r0 + tok of the codes and scales gets
// block `blk`; `live` tokens are written (the last block of a row also clears
// the row's pad bytes).
template <typename T, typename Run>
__device__ __forceinline__ void quantize_tokens(Run run, uint8_t* codes, uint8_t* scales, int64_t r0, int64_t blk,
                                                int64_t code_pitch, int pitch, int live, bool last_block) {
  constexpr int LPT = static_cast<int>(sizeof(T));        // 2, or 4 for FP32
  constexpr int EPL = 32 / LPT;                           // elements per lane
  constexpr int EPR = 16 / static_cast<int>(sizeof(T));   // elements per run
  const int lane = threadIdx.x & 31;
  const int tok = lane / LPT, part = lane % LPT;
  float v[EPL];
  uint32_t amax = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint4 raw = *reinterpret_cast<const uint4*>(run(tok, 2 * part + q));
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < EPR; ++i) {
      v[q * EPR + i] = to_f32(e[i]);
      amax = max(amax, __float_as_uint(v[q * EPR + i]) & 0x7FFFFFFFu);
    }
  }
#pragma unroll
  for (int off = 1; off < LPT; off <<= 1) amax = max(amax, __shfl_xor_sync(FULL_MASK, amax, off));
  const uint32_t byte = mx_scale_byte(amax);
  const float s = mx_inv_scale(byte);
  uint32_t w[EPL / 8];
#pragma unroll
  for (int q = 0; q < EPL / 8; ++q) {
    float e8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e8[i] = v[q * 8 + i] * s;
    w[q] = byte == 255u ? 0u : mx_pack8(e8);
  }
  if (tok >= live) return;
  uint8_t* c = codes + (r0 + tok) * code_pitch + blk * 16 + part * (EPL / 2);
  if constexpr (EPL == 16) *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(c) = w[0];
  if (part == 0) {
    uint8_t* sp = scales + (r0 + tok) * pitch;
    sp[blk] = static_cast<uint8_t>(byte);
    if (last_block)
      for (int p = static_cast<int>(blk) + 1; p < pitch; ++p) sp[p] = 0;
  }
}

template <typename T, bool GATE_UP>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    experts_mx_kernel(const __grid_constant__ MxMaps maps, const __grid_constant__ MxArgs args) {
  using C = MxCfg;
  constexpr int STAGES = C::STAGES;
  constexpr int SF_STAGES = C::SF_STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::SMEM_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* sf_full = empty + STAGES;
  uint64_t* sf_empty = sf_full + SF_STAGES;
  uint64_t* sf_ready = sf_empty + SF_STAGES;  // [SLOTS]
  uint64_t* tfull = sf_ready + C::SLOTS;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::SMEM_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::SMEM_MISC + 4);
  uint32_t* issued_stages = reinterpret_cast<uint32_t*>(smem + C::SMEM_MISC + 8);  // producer's, scale loader's
  uint32_t* tile_start = reinterpret_cast<uint32_t*>(smem + C::SMEM_TILES);  // [E + 1]
  uint32_t* offs = tile_start + args.E + 1;                                   // [E + 1]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < SF_STAGES; ++s) {
      mbar_init(&sf_full[s], 1 + 32);  // the weights' expect_tx, and each lane's copies of the tokens' words
      mbar_init(&sf_empty[s], 4);
    }
    for (int s = 0; s < C::SLOTS; ++s) mbar_init(&sf_ready[s], 4);
    mbar_init(tfull, 1);
    mbar_init(tempty, NUM_EPI_WARPS);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&maps.a0);
    if (GATE_UP) tma_prefetch_desc(&maps.a1);
    for (int i = 0; i < NUM_BOXES; ++i) tma_prefetch_desc(&maps.b[i]);
    if (sizeof(T) == 2 && args.out != nullptr) tma_prefetch_desc(&maps.out);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  // From here on the kernel reads what earlier kernels wrote.
  grid_dependency_wait();
  if (warp == 0)
    build_mx_prefix(args.offsets, args.E, args.rows_total, args.n_wblocks, tile_start, offs);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // The cap keeps a corrupt offsets array from producing an endless tile loop.
  const uint32_t total = min(tile_start[args.E], args.tile_cap);
  const int k_blocks = (args.K + BK - 1) / BK;
  const int k_words = (args.K + 127) / 128;  // 32-bit scale words of a row

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0;
      bool ok = true;
      for (uint32_t tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
        const MxTile tc = decode_mx_tile(tile, tile_start, args.E, args.n_wblocks, offs);
        const uint32_t tx = static_cast<uint32_t>(2 * A_BYTES + tc.n_tok * ROW_BYTES);
        const int row = tc.w * (GATE_UP ? BM : 2 * BM);
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, args.status, ST_PRODUCER_EMPTY,
                                 WAIT_LIMIT_NS)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + stage * C::STAGE_BYTES;
          const int k0 = kb * ROW_BYTES;
          mbar_arrive_expect_tx(&full[stage], tx);
          tma_load_3d(st, &maps.a0, &full[stage], k0, row, tc.e);  // down: both 128-row blocks in one box
          if (GATE_UP) tma_load_3d(st + A_BYTES, &maps.a1, &full[stage], k0, row, tc.e);
          uint8_t* b_dst = st + C::OFF_B;
          int r = 0;
#pragma unroll
          for (int i = 0; i < NUM_BOXES; ++i) {  // 128, 64, 32, 16 rows: the binary digits of n_tok
            if ((tc.n_tok & (128 >> i)) != 0) {
              tma_load_2d(b_dst + r * ROW_BYTES, &maps.b[i], &full[stage], k0, static_cast<int>(tc.row0) + r);
              r += 128 >> i;
            }
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      launch_dependents();  // this CTA issues no more loads
      issued_stages[0] = issued;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (lane == 0) {
      uint32_t n = 0;  // stages consumed
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t tile = blockIdx.x; ok && tile < total; tile += gridDim.x, ++it) {
        const MxTile tc = decode_mx_tile(tile, tile_start, args.E, args.n_wblocks, offs);
        const uint32_t idesc0 = idesc_mxf4(tc.n_tok, 0), idesc2 = idesc_mxf4(tc.n_tok, 2);
        if (!mbar_wait_bounded(tempty, (it & 1u) ^ 1u, abort_flag, args.status, ST_MMA_TMEM_EMPTY,
                               WAIT_LIMIT_NS)) {
          ok = false;
          break;
        }
        for (int kb = 0; kb < k_blocks; ++kb, ++n) {
          const uint32_t stage = n % STAGES, slot = n % C::SLOTS;
          if (!mbar_wait_bounded(&full[stage], (n / STAGES) & 1u, abort_flag, args.status, ST_MMA_FULL,
                                 WAIT_LIMIT_NS) ||
              !mbar_wait_bounded(&sf_ready[slot], (n / C::SLOTS) & 1u, abort_flag, args.status, ST_MMA_SF_READY,
                                 WAIT_LIMIT_NS)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sf = tmem_base + C::SF_BASE + slot * C::SF_COLS;
          const uint32_t sfb = sf + 8 * ATOMS_K;
          const int left = args.K - kb * BK;  // MMA steps wholly past K are left out
          const uint32_t a0 = smem_u32(smem + stage * C::STAGE_BYTES), a1 = a0 + A_BYTES, b = a0 + C::OFF_B;
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k) {
            if (k * UMMA_K < left) {
              const uint32_t accum = (kb > 0 || k > 0) ? 1u : 0u;
              const uint32_t id = (k & 1) != 0 ? idesc2 : idesc0;
              const uint64_t bd = sdesc_kmajor_sw128(b + k * (UMMA_K / 2));
              const uint32_t sb = sfb + 4 * (k >> 1) * C::GROUPS;
              umma_mxf4(tmem_base, sdesc_kmajor_sw128(a0 + k * (UMMA_K / 2)), bd, id, sf + 4 * (k >> 1), sb, accum);
              umma_mxf4(tmem_base + TBN, sdesc_kmajor_sw128(a1 + k * (UMMA_K / 2)), bd, id,
                        sf + 4 * ATOMS_K + 4 * (k >> 1), sb, accum);
            }
          }
          umma_commit(&empty[stage]);
        }
        if (!ok) break;
        umma_commit(tfull);
      }
      // Every copy and MMA issued above completes before TMEM is released.
      umma_commit(drain);
      mbar_wait_bounded(drain, 0, nullptr, args.status, ST_MMA_DRAIN, WAIT_LIMIT_NS);
    }
    __syncwarp();
  } else if (warp < FIRST_SCALE_WARP) {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - 2;
    const int quad = warp & 3;                  // TMEM lanes 32*quad ..
    const int group = ew >> 2;                  // takes 16-token chunks group, group + 4, ...
    uint8_t* xp = smem + C::SMEM_XPOSE + ew * XPOSE_BYTES;
    const uint32_t xp_u32 = smem_u32(xp);
    uint32_t it = 0;
    for (uint32_t tile = blockIdx.x; tile < total; tile += gridDim.x, ++it) {
      const MxTile tc = decode_mx_tile(tile, tile_start, args.E, args.n_wblocks, offs);
      const bool ok = mbar_wait_bounded(tfull, it & 1u, abort_flag, args.status, ST_EPI_TMEM_FULL,
                                        WAIT_LIMIT_NS);
      if (!__all_sync(FULL_MASK, ok)) break;  // tcgen05.ld is warp-collective: the whole warp goes on or stops
      tc_fence_after();
      const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
      const int64_t colA = static_cast<int64_t>(tc.w) * (GATE_UP ? BM : 2 * BM) + quad * 32;
      // Rows of the tile that exist in the buffers (all of them, for valid offsets).
      const int live = tc.row0 < args.rows_total
                           ? static_cast<int>(min(static_cast<uint32_t>(tc.rows), args.rows_total - tc.row0)) : 0;
      constexpr int GROUPS = NUM_EPI_WARPS / 4;
      // The accumulators may be overwritten once every warp has read its part.
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty);
      };
      if constexpr (sizeof(T) == 2) {
        // A chunk is read as fragments of 16 channels x 16 tokens and packed,
        // token pairs in a word; it leaves through the warp's buffer, transposed
        // by stmatrix into token rows of 32 channels (64 bytes, 16-byte runs in
        // the 64-byte swizzle: the stores and both kinds of reads below are free
        // of bank conflicts). The last HOLD chunks are all read before any of
        // them is stored: the next tile's MMAs start after the reads, and the
        // transposes and stores overlap them (gate/up of 16384 rows: 672 -> 639
        // us; down has twice the words a chunk, and holding all four spills).
        constexpr int CHUNKS = (TBN / EPI_TOKENS + GROUPS - 1) / GROUPS;
        constexpr int BLKS = GATE_UP ? 1 : 2;
        constexpr int HOLD = GATE_UP ? CHUNKS : 2;
        auto read_chunk = [&](int c0, uint32_t (&m)[BLKS][2][4]) {
          uint32_t f0[2][8], f1[2][8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = t_lane + (static_cast<uint32_t>(16 * h) << 16) + static_cast<uint32_t>(c0);
            tmem_ld_16x256b_x2(at, f0[h]);
            tmem_ld_16x256b_x2(at + TBN, f1[h]);
          }
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int r = 4 * i + 2 * (q & 1);
              const float a0 = __uint_as_float(f0[q >> 1][r]), a1 = __uint_as_float(f0[q >> 1][r + 1]);
              const float b0 = __uint_as_float(f1[q >> 1][r]), b1 = __uint_as_float(f1[q >> 1][r + 1]);
              if constexpr (GATE_UP) {
                m[0][i][q] = pack2<T>(mx_silu<T>(a0) * b0, mx_silu<T>(a1) * b1);
              } else {
                m[0][i][q] = pack2<T>(a0, a1);
                m[BLKS - 1][i][q] = pack2<T>(b0, b1);
              }
            }
          }
        };
        auto store_chunk = [&](int c0, const uint32_t (&m)[BLKS][2][4]) {
          const int64_t row = static_cast<int64_t>(tc.row0) + c0;
#pragma unroll
          for (int blk = 0; blk < BLKS; ++blk) {
            const int64_t col0 = colA + blk * BM;
            if (col0 >= args.n_out) continue;  // n_out is a multiple of 32: the warp's block is in or out
            if (lane == 0) bulk_wait_read_all();  // the buffer's last bulk store has read it
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int tok = 8 * i + (lane & 7);
              stmatrix_x4_trans(xp_u32 + static_cast<uint32_t>(tok * 64 + (((lane >> 3) ^ (tok >> 1)) & 3) * 16),
                                m[blk][i][0], m[blk][i][1], m[blk][i][2], m[blk][i][3]);
            }
            const bool full_chunk = args.out != nullptr && c0 + EPI_TOKENS <= live;
            if (full_chunk) fence_proxy_async_smem();
            __syncwarp();
            if (full_chunk) {
              // Every token is the tile's: one tensor store.
              if (lane == 0) {
                tma_store_2d(&maps.out, xp_u32, static_cast<int>(col0), static_cast<int>(row));
                bulk_commit_group();
              }
            } else if (args.out != nullptr) {
              // The rows after the tile's are another expert's.
              const int part = lane & 3;
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const int j = p * 8 + (lane >> 2);
                if (c0 + j < live)
                  reinterpret_cast<uint4*>(static_cast<T*>(args.out) + (row + j) * args.n_out + col0)[part] =
                      *reinterpret_cast<const uint4*>(xp + j * 64 + ((part ^ (j >> 1)) & 3) * 16);
              }
            }
            if (GATE_UP && args.q_codes != nullptr)
              quantize_tokens<T>([&](int tok, int q) { return xp + tok * 64 + ((q ^ (tok >> 1)) & 3) * 16; },
                                 args.q_codes, args.q_scales, row, col0 / MX_BLOCK, args.n_out / 2, args.q_pitch,
                                 live - c0, col0 + MX_BLOCK >= args.n_out);
            __syncwarp();
          }
        };
        auto chunk_at = [&](int c) { return EPI_TOKENS * (group + GROUPS * c); };
        const int mine = (tc.n_tok / EPI_TOKENS - group + GROUPS - 1) / GROUPS;  // this warp's chunks
        const int first_held = mine > HOLD ? mine - HOLD : 0;
#pragma unroll 1
        for (int c = 0; c < first_held; ++c) {
          uint32_t m[BLKS][2][4];
          read_chunk(chunk_at(c), m);
          store_chunk(chunk_at(c), m);
        }
        uint32_t held[HOLD][BLKS][2][4];
#pragma unroll
        for (int c = 0; c < HOLD; ++c)
          if (first_held + c < mine) read_chunk(chunk_at(first_held + c), held[c]);
        release();
#pragma unroll
        for (int c = 0; c < HOLD; ++c)
          if (first_held + c < mine) store_chunk(chunk_at(first_held + c), held[c]);
      } else {
        for (int c0 = EPI_TOKENS * group; c0 < tc.n_tok; c0 += EPI_TOKENS * GROUPS) {
          const int64_t row = static_cast<int64_t>(tc.row0) + c0;
          // FP32: lane = output channel, register = token, 8 tokens at a time
          // through the buffer, stored lane by lane. The accumulators are
          // released after the last store (held, they would be twice the words
          // of the 16-bit outputs), so the stores overlap no MMA either:
          // gate/up of 16384 rows 758 us against 646 in BF16, the down product
          // of 32768 rows, E=128, H=2048, I=768 74 against 54.
          uint32_t v0[16], v1[16];
          tmem_ld_32x32b_x16(t_lane + static_cast<uint32_t>(c0), v0);
          tmem_ld_32x32b_x16(t_lane + TBN + static_cast<uint32_t>(c0), v1);
          tmem_ld_wait();
          float* xf = reinterpret_cast<float*>(xp);
#pragma unroll
          for (int blk = 0; blk < (GATE_UP ? 1 : 2); ++blk) {
            const int64_t col0 = colA + blk * BM;
            const bool col_ok = col0 < args.n_out;
#pragma unroll
            for (int t0 = 0; t0 < EPI_TOKENS; t0 += 8) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float a = __uint_as_float(v0[t0 + j]), b = __uint_as_float(v1[t0 + j]);
                xf[j * 32 + lane] = GATE_UP ? mx_silu<T>(a) * b : (blk == 0 ? a : b);
              }
              __syncwarp();
              if (args.out != nullptr && col_ok) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                  const int j = p * 4 + (lane >> 3);
                  if (c0 + t0 + j < live)
                    reinterpret_cast<uint4*>(static_cast<T*>(args.out) + (row + t0 + j) * args.n_out + col0)[lane & 7] =
                        *reinterpret_cast<const uint4*>(xf + j * 32 + (lane & 7) * 4);
                }
              }
              if (GATE_UP && args.q_codes != nullptr && col_ok)
                quantize_tokens<T>([&](int tok, int q) { return xp + tok * 128 + q * 16; }, args.q_codes,
                                   args.q_scales, row + t0, col0 / MX_BLOCK, args.n_out / 2, args.q_pitch,
                                   live - c0 - t0, col0 + MX_BLOCK >= args.n_out);
              __syncwarp();
            }
          }
        }
        release();
      }
    }
    if (lane == 0) bulk_wait_all();  // the stores have left shared memory and are done
  } else if (warp < LOAD_WARP) {
    // ------------------------------------------------------------ scales, shared -> TMEM
    // Each warp writes its 32 lanes' quarter of every stage's scale buffer (the
    // MMA wants the atoms' 32 rows repeated in the four quarters).
    const uint32_t quad_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t n = 0;
    bool ok = true;
    for (uint32_t tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
      for (int kb = 0; kb < k_blocks; ++kb, ++n) {
        const uint32_t ss = n % SF_STAGES;
        ok = mbar_wait_bounded(&sf_full[ss], (n / SF_STAGES) & 1u, abort_flag, args.status, ST_SCALE_FULL,
                               WAIT_LIMIT_NS);
        ok = __all_sync(FULL_MASK, ok);
        if (!ok) break;
        // Atoms in the order of the buffer's columns: SFA0 and SFA1 by K
        // atom (they lie interleaved), then SFB.
        const uint8_t* src = smem + C::SMEM_SF + ss * C::SF_BYTES + lane * 16;
        uint4 v[C::SF_COLS / 4];
#pragma unroll
        for (int a = 0; a < ATOMS_K; ++a) {
          v[a] = *reinterpret_cast<const uint4*>(src + 2 * a * ATOM);
          v[ATOMS_K + a] = *reinterpret_cast<const uint4*>(src + (2 * a + 1) * ATOM);
        }
#pragma unroll
        for (int i = 2 * ATOMS_K; i < C::SF_COLS / 4; ++i) v[i] = *reinterpret_cast<const uint4*>(src + i * ATOM);
        if (n >= static_cast<uint32_t>(C::SLOTS)) {
          // The buffer's last readers: the MMAs of stage n - SLOTS.
          const uint32_t p = n - C::SLOTS;
          ok = mbar_wait_bounded(&empty[p % STAGES], (p / STAGES) & 1u, abort_flag, args.status, ST_SCALE_SLOT,
                                 WAIT_LIMIT_NS);
          ok = __all_sync(FULL_MASK, ok);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t sf = tmem_base + C::SF_BASE + (n % C::SLOTS) * C::SF_COLS + quad_lane;
#pragma unroll
        for (int i = 0; i < C::SF_COLS / 8; ++i) tmem_st_32x32b_x8(sf + 8 * i, v[2 * i], v[2 * i + 1]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sf_ready[n % C::SLOTS]);
          // Only now is the ring slot free: the stores have used the loads'
          // results. Released right after the loads were issued, a slot could
          // be overwritten under them.
          mbar_arrive(&sf_empty[ss]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ scales, global -> shared
    // Lane 0 takes a stage's weight atoms with one bulk copy, all lanes the
    // tokens' words: word a of token t (its four scale bytes for K elements
    // 256 kb + 128 a ..) goes to atom (a, t / 128). Bytes past K / 32 and rows
    // past the tile are filled with 0, never read. (One warp keeps up: two or
    // four measured the same or slower, each a further poller of barriers.)
    uint32_t n = 0;
    bool ok = true;
    for (uint32_t tile = blockIdx.x; ok && tile < total; tile += gridDim.x) {
      const MxTile tc = decode_mx_tile(tile, tile_start, args.E, args.n_wblocks, offs);
      const uint8_t* sfa = args.sfa + (static_cast<int64_t>(tc.e) * args.n_wblocks + tc.w) * k_words * (2 * ATOM);
      // This lane's tokens lane, lane + 32, ...: their rows, or NULL past the tile's.
      constexpr int TPL = (TBN + 31) / 32;
      const uint8_t* rows[TPL];
#pragma unroll
      for (int i = 0; i < TPL; ++i) {
        const int tok = lane + 32 * i;
        const uint32_t row = tc.row0 + static_cast<uint32_t>(tok);
        const bool in = tok < tc.rows && row < args.rows_total;
        rows[i] = in ? args.sfb + static_cast<int64_t>(row) * args.sfb_pitch : nullptr;
      }
      for (int kb = 0; kb < k_blocks; ++kb, ++n) {
        const uint32_t ss = n % SF_STAGES;
        ok = mbar_wait_bounded(&sf_empty[ss], ((n / SF_STAGES) & 1u) ^ 1u, abort_flag, args.status, ST_LOADER_EMPTY,
                               WAIT_LIMIT_NS);
        ok = __all_sync(FULL_MASK, ok);
        if (!ok) break;
        uint8_t* slot = smem + C::SMEM_SF + ss * C::SF_BYTES;
        if (lane == 0) {
          // The last stage may hold fewer atoms than the others (the MMA
          // steps past K are left out).
          const uint32_t bytes = static_cast<uint32_t>(min(ATOMS_K, k_words - kb * ATOMS_K)) * (2 * ATOM);
          mbar_arrive_expect_tx(&sf_full[ss], bytes);
          bulk_load(slot, sfa + static_cast<int64_t>(kb) * SFA_BYTES, bytes, &sf_full[ss]);
        }
        const uint32_t dst = smem_u32(slot) + SFA_BYTES + static_cast<uint32_t>(lane * 16);
#pragma unroll
        for (int i = 0; i < TPL; ++i) {
          if (32 * i >= tc.n_tok) break;
#pragma unroll
          for (int a = 0; a < ATOMS_K; ++a) {
            const int byte0 = (kb * ATOMS_K + a) * 4;
            const int valid = rows[i] != nullptr ? max(0, min(4, args.sf_blocks - byte0)) : 0;
            cp_async_4(dst + static_cast<uint32_t>((a * C::GROUPS + i / 4) * ATOM + (i % 4) * 4),
                       valid > 0 ? rows[i] + byte0 : args.sfb, static_cast<uint32_t>(valid));
          }
        }
        cp_async_mbar_arrive_noinc(&sf_full[ss]);
      }
    }
    cp_async_wait_all();  // this lane's copies of token scales; the bulk copies of weight scales are waited for below
    if (lane == 0) issued_stages[1] = n;
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag != 0) {
    // A role gave up: the copies that nobody waited for land before the block
    // exits (they would write shared memory, and signal barriers, that are the
    // next block's). Every lane of the scale loader has arrived on each stage
    // that its lane 0 armed: it leaves its loop before arming, as one warp.
    if (threadIdx.x == 0)
      drain_ring(issued_stages[0], STAGES, [&](uint32_t slot, uint32_t parity) {
        mbar_wait_bounded(&full[slot], parity, nullptr, args.status, ST_PRODUCER_DRAIN, WAIT_LIMIT_NS);
      });
    if (threadIdx.x == 32 * LOAD_WARP)
      drain_ring(issued_stages[1], SF_STAGES, [&](uint32_t slot, uint32_t parity) {
        mbar_wait_bounded(&sf_full[slot], parity, nullptr, args.status, ST_LOADER_DRAIN, WAIT_LIMIT_NS);
      });
    __syncwarp();
  }
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

// [rows, n] 16-bit outputs, boxes of 32 columns x EPI_TOKENS rows with the 64-byte swizzle.
bool encode_out(CUtensorMap* m, moe_dtype dtype, void* ptr, uint64_t n, uint64_t rows) {
  auto fn = encode_fn_mx();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {n, rows};
  const cuuint64_t strides[1] = {n * 2};
  const cuuint32_t box[2] = {32, EPI_TOKENS};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, dtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, ptr, dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [E, rows, row_bytes] codes, box 128 bytes (one swizzle atom) x box_rows x 1.
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

template <typename T, bool GATE_UP>
cudaError_t launch_mx(const MxMaps& maps, MxArgs args, int64_t rows, int num_sms, cudaStream_t stream) {
  auto kern = experts_mx_kernel<T, GATE_UP>;
  constexpr int SMEM_BYTES = MxCfg::SMEM_BYTES;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (err != cudaSuccess) return err;
  // At most ceil(rows_e / TBN) token tiles per expert.
  const int64_t cap = (rows / TBN + (rows < args.E ? rows : args.E)) * args.n_wblocks;
  args.tile_cap = static_cast<uint32_t>(cap < 0xFFFFFFFFll ? cap : 0xFFFFFFFFll);
  const int grid = static_cast<int>(cap < num_sms ? cap : num_sms);
  return launch_dependent(kern, dim3(grid), dim3(NUM_THREADS), SMEM_BYTES, stream, maps, args);
}

// What a launch needs beside MxArgs: the operands' pointers for its maps.
struct MxOperands {
  bool gate_up;
  const void* w0;      // gate or down codes [E, N, K / 2]
  const void* w1;      // up codes
  const void* tokens;  // [rows, K / 2]
};

template <typename T>
cudaError_t stage_t(const MxOperands& op, const MxArgs& args, int64_t rows, int num_sms, cudaStream_t stream,
                    const char** why) {
  const uint64_t kb = static_cast<uint64_t>(args.K / 2), N = static_cast<uint64_t>(args.n_out);
  const uint64_t E = static_cast<uint64_t>(args.E);
  MxMaps maps;
  bool ok = encode_codes(&maps.a0, op.w0, kb, N, E, op.gate_up ? BM : 2 * BM, 3);
  maps.a1 = maps.a0;
  if (op.gate_up) ok = ok && encode_codes(&maps.a1, op.w1, kb, N, E, BM, 3);
  for (int i = 0; i < NUM_BOXES; ++i)
    ok = ok && encode_codes(&maps.b[i], op.tokens, kb, static_cast<uint64_t>(rows), 1, 128u >> i, 2);
  maps.out = maps.a0;
  if (sizeof(T) == 2 && args.out != nullptr)
    ok = ok && encode_out(&maps.out, std::is_same<T, __half>::value ? MOE_F16 : MOE_BF16, args.out, N,
                          static_cast<uint64_t>(rows));
  if (!ok) {
    *why = "cuTensorMapEncodeTiled rejected a tensor map";
    return cudaErrorInvalidValue;
  }
  return op.gate_up ? launch_mx<T, true>(maps, args, rows, num_sms, stream)
                    : launch_mx<T, false>(maps, args, rows, num_sms, stream);
}

}  // namespace

// Weight blocks per expert of a stage: 128 gate and 128 up rows, or 256 down
// rows; each has two 128-row atoms' worth of scales per K block.
int64_t mx_weight_blocks(bool gate_up, int64_t R) { return gate_up ? (R + BM - 1) / BM : (R + 2 * BM - 1) / (2 * BM); }

size_t mx_weight_scale_bytes(bool gate_up, int64_t E, int64_t R, int64_t K) {
  return static_cast<size_t>(E) * static_cast<size_t>(mx_weight_blocks(gate_up, R)) *
         static_cast<size_t>((K + 127) / 128) * (2 * ATOM);
}

cudaError_t launch_experts_mx(const MxWeights& w, bool gate_up, const void* codes, const void* scales,
                              const uint32_t* offsets, int E, int64_t rows, int64_t H, int64_t I, moe_dtype out_dtype,
                              void* out, void* q_codes, void* q_scales, int num_sms, cudaStream_t stream,
                              const char** why) {
  if (rows == 0) return cudaSuccess;
  const int64_t K = gate_up ? H : I;
  const int64_t N = gate_up ? I : H;
  MxArgs a{};
  cudaError_t err = device_status_ptr(&a.status);
  if (err != cudaSuccess) return err;
  a.offsets = offsets;
  a.sfa = static_cast<const uint8_t*>(gate_up ? w.gate_up_sf : w.down_sf);
  a.sfb = static_cast<const uint8_t*>(scales);
  a.sfb_pitch = static_cast<int>(mx_scale_pitch(K));
  a.sf_blocks = static_cast<int>(K / MX_BLOCK);
  a.E = E;
  a.n_wblocks = static_cast<int>(mx_weight_blocks(gate_up, N));
  a.K = static_cast<int>(K);
  a.n_out = static_cast<int>(N);
  a.rows_total = static_cast<uint32_t>(rows);
  a.out = out;
  a.q_codes = static_cast<uint8_t*>(q_codes);
  a.q_scales = static_cast<uint8_t*>(q_scales);
  a.q_pitch = static_cast<int>(mx_scale_pitch(N));
  const MxOperands op{gate_up, gate_up ? w.gate : w.down, w.up, codes};
  if (out_dtype == MOE_F32) return stage_t<float>(op, a, rows, num_sms, stream, why);
  if (out_dtype == MOE_F16) return stage_t<__half>(op, a, rows, num_sms, stream, why);
  return stage_t<__nv_bfloat16>(op, a, rows, num_sms, stream, why);
}

}  // namespace moe
