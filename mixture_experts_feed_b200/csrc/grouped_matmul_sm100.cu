// Grouped matrix products (moe_grouped_matmul and its two gradients) on the
// sm_100a tensor cores: out[i, j] = sum_r P[i, r] Q[j, r] for ragged groups
// of rows, bf16 or fp16 operands, fp32 accumulators in tensor memory.
//
//             i (output row)     j (contiguous)    r (summed)
//   forward   row of the group   n index           k index
//   dgrad     row of the group   k index           n index
//   wgrad     n index            k index           row of the group
//
// The MMA's M side is j and its N side is i: a CTA pair (tcgen05
// cta_group::2) computes 256 j x up to 256 i, the accumulator holding the
// output transposed (lane = j, column = i).  N may be any multiple of 32, so
// the ragged side pads to 32 rows instead of a whole 128- or 256-row tile: a
// group of 40 rows costs a 64-wide MMA, a decoded token a 32-wide one, and
// the weights stream through the M side at full width either way.  A group's
// rows are cut into ceil(rows / 256) tiles of even height.
//
// Operands come by TMA with the 128-byte swizzle in whichever order they lie
// in memory: r contiguous ("K-major": boxes of 64 r x rows) or j / i
// contiguous ("MN-major": boxes of 64 j x 64 r, two per tile side), told to
// the MMA by its descriptors.  No transposed copy exists anywhere.
//   forward  M: W[e] K-major    N: a K-major
//   dgrad    M: W[e] MN-major   N: dout K-major
//   wgrad    M: a MN-major      N: dout MN-major
//
// wgrad sums over a group's rows, whose last block of 64 may run into the
// next group's rows (or rows that belong to nobody, which may hold NaN).
// That block's loads complete on a barrier of their own CTA; a warp of each
// CTA then overwrites the foreign rows up to the next multiple of 16 with
// zeros in shared memory, for both operands, and the MMA runs that many
// 16-row steps.
//
// The accumulator truncates instead of rounding at every step, an error that
// grows with the chain and always leans toward zero (2-norm, random normal
// operands: 2.3e-7 for chains of 256 terms, 4.7e-7 for 512, 1.0e-6 for 1024,
// 6.7e-6 for 6144; a library product in fp32 has 1.6e-7 to 6e-7.  Products of
// one sign: 3e-6 for 512, and 4.2e-4 for 65536, a whole half step of fp16).
// One chain is kept to 512 terms (kChain blocks of 64), and the chains of a tile
// are added in fp32 registers by the warps that store it, in order, for every
// type of output.  Against one chain of any length that takes 1.5% more on 16-bit
// forward products (24576 rows of 64 experts, 2048 x 2048: 223.7 us / 220.4) and
// 1% on their weight gradients; chains of 256 cost 6% on the largest fp32 input
// gradient.
//
// Few tiles with a long sum (the weight gradient of one large expert, a
// product of few rows with a long k) would leave most pairs idle.  Such tiles are cut
// along r into pieces, each a tile of its own whose accumulator goes to a slot
// of the workspace, and a second kernel adds a tile's slots in order:
// reproducible, where adds to memory would not be.  Measured (us, cut / whole):
// dW of one expert of 16384 rows, 256 x 256, 19 / 79; of 8192 rows, 1024 x 1024,
// 29 / 44; 65536 rows all in one of 64 experts, 512 x 512, 54 / 303; 249 rows,
// k = 4096, n = 1024, 18 / 25.  Bound now by launches and drain, the loads, and the
// slots through L2.
//
// Roles (one CTA an SM): warp 0 loads, warp 1 allocates tensor memory and
// (rank 0) issues the MMAs, warp 10 works the tiles out, warp 11 mends wgrad's
// partial blocks, warps 2..9 store (through staging boxes and TMA stores;
// accumulation into fp32 weight gradients is TMA's add); two accumulators let
// the stores of one tile overlap the MMAs of the next.  Every wait is bounded.
//
// What bounds it.  A block of 64 r costs a pair 512 clocks of MMA at N = 256
// and brings 32 KB to each SM, about what the TMA unit moves in that time (64
// bytes a clock, a row of 128 bytes at a time): 8192^3 in bf16 keeps the tensor
// pipe busy 95% of a launch's 0.97 M clocks.  To get there the loading and issuing
// warps run converged and elect a lane for the instruction itself (with one lane
// in the loop every operand went through the vector registers, 730 clocks a
// block), nothing but the MMAs' operands lies between two tiles (tiles come from a
// queue), and accumulators are handed back with a light arrival.  From there
// the 1 kW power limit sets the clock.  Measured on B200s, back to back (SM
// clock 1.0 to 1.3 GHz): 8192^3 1279 TFLOP/s (the library product 1343 to 1366);
// 65536 rows of 128 experts, n = 4096, k = 6144, fp32 dx, 947 to 990 TFLOP/s at
// 2.5 TB/s; 24576 rows of 64 experts, n = k = 2048: forward 892 to 920, dW 860 to
// 893 TFLOP/s at 3.1 TB/s.  DRAM traffic is the algorithm's (forward: 638 MB read
// for 637, dW 201 for 201).  Six decoded rows (50 MB of weights) take 15 us.
#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "grouping.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int TM = 256;                  // j per tile (a CTA pair; 128 a CTA)
constexpr int TN = 256;                  // i per tile, at most
constexpr int BK = 64;                   // r per stage
constexpr int SIDE_BYTES = 128 * BK * 2; // one operand of a stage in one CTA
constexpr int STAGE_BYTES = 2 * SIDE_BYTES;
constexpr int STAGES = 6;                // or one fewer beside large tables (many experts)
constexpr int EPI_WARPS = 8;              // two per quarter of the tensor memory's lanes
constexpr int SCHED_WARP = 2 + EPI_WARPS;
constexpr int FIX_WARP = SCHED_WARP + 1; // wgrad's last blocks
__host__ __device__ constexpr int num_threads(int form) { return 32 * (form == kWgrad ? FIX_WARP + 1 : FIX_WARP); }
constexpr int OUT_BYTES = 4096;          // staging of an epilogue warp (16-bit: 8 KB for two warps)
constexpr uint32_t TMEM_COLS = 512;      // two accumulators of 256 columns
constexpr int TQ = 8;                    // slots of the tile queue
constexpr int kBand = 8;                 // i tiles per band (tile order)
constexpr int kChain = 8;                // blocks of 64 per accumulation chain
constexpr int kMaxSmem = 232448;         // shared memory a block can have
constexpr int kSplitUnits = 74;          // CTA pairs that pieces are made for
constexpr int kMinPiece = 8;             // blocks of 64 r of a piece, at least
constexpr int kMinGain = 24;             // blocks that cutting saves the longest tile, at least
constexpr int64_t kSkewedRows = 16384;   // wgrad: rows from which skewed groups are provided for
constexpr int kCutWord = 32;             // word of the status region behind the status and the counters
constexpr int kJoinRows = 4;             // i of a step of the joining kernel

// What the tables are made of.
struct Shape {
  const int32_t* offsets;
  int E, rows_cap;
  int n_i, n_j, n_r;     // sizes of i, j, r (0 where it is the group's rows)
  int accumulate;
  int units;             // split products: CTA pairs of the launch
  int slot_i, slot_j;    // split products: a piece's slot [slot_i][slot_j] of fp32
  int32_t* cut;          // split products: where the first kernel says how many slots it filled
};

struct alignas(64) ProductParams : Shape {
  CUtensorMap tmM;       // M side
  CUtensorMap tmN[4];    // N side: boxes of 128, 64, 32 and 16 rows (wgrad: [0] alone)
  CUtensorMap tmOut;     // output [depth][i][j]: boxes of 64 j x 64 i (16-bit) or 32 x 32 (fp32)
  CUtensorMap tmOut32;   // 16-bit: boxes of 64 j x 32 i
  CUtensorMap tmParts;   // split products: the slots [slots x slot_i][slot_j], boxes of 32 x 32
  int32_t* status;
  void* out;
  uint32_t fmt;          // operand format bits of the MMA descriptor
  int stages;            // pipeline stages
};

struct Smem {
  // full[STAGES], empty[STAGES], tail[STAGES], tfull[2], tempty[2], drain, tq[TQ], tqe[TQ], pair[4]
  static constexpr int kNumBars = 3 * STAGES + 9 + 2 * TQ;
  // the stages, 4 KB of staging a warp, the tile queue, the barriers, then
  // tmem base, abort, bad, piece, then s_off[E + 1], s_tile[E + 1] (split: s_slot[E + 1])
  static constexpr int kFixed = TQ * 32 + kNumBars * 8 + 16;
  static int bytes(int E, int stages, bool split) {
    return 1024 + stages * STAGE_BYTES + EPI_WARPS * OUT_BYTES + kFixed + (split ? 12 : 8) * (E + 1);
  }
};

__host__ __device__ __forceinline__ int tiles_over(int n, int t) { return (n + t - 1) / t; }

// Height of a side of `n` cut into tiles of at most TN: even, a multiple of 32.
__host__ __device__ __forceinline__ int even_height(int n) {
  const int t = tiles_over(n, TN);
  return (tiles_over(n, t > 0 ? t : 1) + 31) & ~31;
}

// Warp: s_off = the checked offsets, s_tile = exclusive prefix of tile counts.
template <int FORM>
__device__ __forceinline__ void build_tables(const Shape& p, int* s_off, int* s_tile, int* bad) {
  const int lane = threadIdx.x & 31;
  load_offsets(p.offsets, p.E, p.rows_cap, s_off, bad);
  const int ct = tiles_over(p.n_j, TM);
  int carry = 0;
  if (lane == 0) s_tile[0] = 0;
  for (int base = 0; base < p.E; base += 32) {
    const int e = base + lane;
    int cnt = 0;
    if (e < p.E) {
      const int rows = s_off[e + 1] - s_off[e];
      if (FORM == kWgrad) cnt = p.accumulate && rows == 0 ? 0 : tiles_over(p.n_i, TN) * ct;
      else cnt = tiles_over(rows, TN) * ct;
    }
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (e < p.E) s_tile[e + 1] = carry + incl;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
}

// Warp: the tables of a split product.  A tile of group e sums over
// group_blocks(e) blocks of r; in ceil(blocks / *s_piece) pieces of even
// length.  Pieces are as long as every pair's share of all blocks, at least
// kMinPiece, and a little longer where the pieces would otherwise make a
// second round; nothing is cut for less than kMinGain blocks.  s_tile =
// exclusive prefix of the pieces (JOIN: of the tiles of more than one piece),
// s_slot = exclusive prefix of the pieces of such tiles: fewer than 2 x units,
// because every tile in pieces has more blocks than a pair's share.
template <int FORM> __device__ __forceinline__ int group_tiles(const Shape& p, const int* s_off, int e) {
  return tiles_over(FORM == kWgrad ? p.n_i : s_off[e + 1] - s_off[e], TN) * tiles_over(p.n_j, TM);
}
template <int FORM> __device__ __forceinline__ int group_blocks(const Shape& p, const int* s_off, int e) {
  return tiles_over(FORM == kWgrad ? s_off[e + 1] - s_off[e] : p.n_r, BK);
}
template <int FORM, bool JOIN>
__device__ __forceinline__ void build_split_tables(const Shape& p, int* s_off, int* s_tile, int* s_slot,
                                                   int* s_piece, int* bad) {
  const int lane = threadIdx.x & 31;
  load_offsets(p.offsets, p.E, p.rows_cap, s_off, bad);
  int64_t work = 0;
  int live = 0, longest = 0;                               // tiles with blocks, the most blocks of one
  for (int e = lane; e < p.E; e += 32) {
    const int t = group_tiles<FORM>(p, s_off, e), b = group_blocks<FORM>(p, s_off, e);
    work += static_cast<int64_t>(t) * b;
    live += b > 0 ? t : 0;
    longest = max(longest, t > 0 ? b : 0);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    work += __shfl_xor_sync(0xffffffffu, work, d);
    live += __shfl_xor_sync(0xffffffffu, live, d);
  }
  int piece = max(kMinPiece, static_cast<int>((work + p.units - 1) / p.units));
  for (int round = 0; round < 8 && live <= p.units; ++round) {
    int pieces = 0;
    for (int e = lane; e < p.E; e += 32)
      pieces += group_tiles<FORM>(p, s_off, e) * tiles_over(group_blocks<FORM>(p, s_off, e), piece);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) pieces += __shfl_xor_sync(0xffffffffu, pieces, d);
    if (pieces <= p.units) break;
    piece += max(1, piece >> 3);
  }
  if (longest - piece < kMinGain) piece = max(piece, longest);
  int carry = 0, slots = 0;
  if (lane == 0) {
    *s_piece = piece;
    s_tile[0] = 0;
    s_slot[0] = 0;
  }
  for (int base = 0; base < p.E; base += 32) {
    const int e = base + lane;
    int cnt = 0, cut = 0;
    if (e < p.E) {
      const int t = group_tiles<FORM>(p, s_off, e), b = group_blocks<FORM>(p, s_off, e);
      const int pieces = tiles_over(b, piece);
      cut = pieces > 1 ? t * pieces : 0;
      cnt = JOIN ? (pieces > 1 ? t : 0) : FORM == kWgrad && p.accumulate && b == 0 ? 0 : t * max(pieces, 1);
    }
    int incl = cnt, incl_cut = cut;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d), w = __shfl_up_sync(0xffffffffu, incl_cut, d);
      if (lane >= d) { incl += v; incl_cut += w; }
    }
    if (e < p.E) {
      s_tile[e + 1] = carry + incl;
      s_slot[e + 1] = slots + incl_cut;
    }
    carry += __shfl_sync(0xffffffffu, incl, 31);
    slots += __shfl_sync(0xffffffffu, incl_cut, 31);
  }
  __syncwarp();
}

// Group whose run of the prefix table holds `tile`.
__device__ __forceinline__ int find_group(int tile, int E, const int* s_tile) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_tile[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tile `local` of a group of it x jt tiles.  The shorter tile side runs
// innermost (consecutive tiles share the other side's operand from L2); when
// both are long, bands of kBand i tiles, j by j inside a band.
__device__ __forceinline__ void tile_at(int local, int it, int jt, int& i, int& j) {
  if (it > kBand && jt > kBand) {
    const int band = local / (kBand * jt);
    const int in_band = local - band * kBand * jt;
    const int height = min(kBand, it - band * kBand);
    j = in_band / height;
    i = band * kBand + (in_band - j * height);
  } else if (it > jt) {
    i = local / jt;
    j = local - i * jt;
  } else {
    j = local / it;
    i = local - j * it;
  }
}

struct alignas(32) TileInfo {
  int e;         // group
  int row0;      // the group's first row
  int rows;      // its rows
  int i0, j0;    // tile origin (i inside the group for forward and dgrad)
  int ni;        // valid i in the tile
  int mma_n;     // N of its MMAs: ni rounded up to 32
  int blocks;    // blocks of 64 r; -1: no more tiles
};

// Piece `tile` of a split product: the tile's blocks are the piece's, so a piece
// of a weight gradient is a tile of fewer rows; forward and dgrad, which do not
// use `rows`, have the piece's first block there.  Bits 10 and up of e:
// 1 + the piece's slot, or 0 for a tile in one piece.
constexpr int kGroupBits = 10;
template <bool SPLIT> __device__ __forceinline__ int group_of(const TileInfo& t) {
  return SPLIT ? t.e & ((1 << kGroupBits) - 1) : t.e;
}

// Tile `tile` of the launch.
template <int FORM, bool SPLIT>
__device__ __forceinline__ TileInfo tile_info(int tile, const Shape& p, const int* s_off, const int* s_tile,
                                              const int* s_slot, int piece) {
  TileInfo t;
  const int e = find_group(tile, p.E, s_tile);
  t.e = e;
  t.row0 = s_off[e];
  t.rows = s_off[e + 1] - s_off[e];
  const int n_i = FORM == kWgrad ? p.n_i : t.rows;
  const int n_r = FORM == kWgrad ? t.rows : p.n_r;
  const int it = tiles_over(n_i, TN), jt = tiles_over(p.n_j, TM);
  int local = tile - s_tile[e];
  t.blocks = tiles_over(n_r, BK);
  if (SPLIT) {
    const int pieces = tiles_over(t.blocks, piece);
    int first = 0;
    if (pieces > 1) {
      t.e |= (1 + s_slot[e] + local) << kGroupBits;
      const int mine = local / (it * jt);
      local -= mine * it * jt;
      const int each = tiles_over(t.blocks, pieces);      // mine * each < blocks for every piece
      first = mine * each;
      t.blocks = min(each, t.blocks - first);
    }
    if (FORM == kWgrad) {
      t.row0 += first * BK;
      t.rows = min(t.rows - first * BK, t.blocks * BK);
    } else {
      t.rows = first;
    }
  }
  int i, j;
  tile_at(local, it, jt, i, j);
  const int h = even_height(n_i);
  t.i0 = i * h;
  t.j0 = j * TM;
  t.ni = min(h, n_i - t.i0);
  t.mma_n = (t.ni + 31) & ~31;
  return t;
}

// Shared-memory descriptor of an MN-major operand written by TMA boxes of 64
// elements (128 bytes, swizzled) x 64 r, box after box: leading offset = one
// box (8192 bytes, the next 64 elements), stride offset = 8 r (1024 bytes).
__device__ __forceinline__ uint64_t smem_desc_mnmajor_sw128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// mbar_wait for a whole warp that can be late: one lane asks, and sleeps in
// between, so that waiting warps leave the issue slots and the shared-memory
// pipe to the warps that load and issue MMAs.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int32_t* status) {
  int got = 1;
  if ((threadIdx.x & 31) == 0 && !mbar_try_wait(bar, parity)) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (*abort) { got = 0; break; }
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        record_status(status, DEV_WAIT_TIMEOUT);
        *abort = 1;
        got = 0;
        break;
      }
      __nanosleep(100);
    }
  }
  got = __shfl_sync(0xffffffffu, got, 0);
  __syncwarp();                            // the shuffle alone orders no memory
  return got != 0;
}

// mbar_wait by a whole warp that stays converged; `cluster`: with acquire at
// cluster scope, for what threads of the other CTA wrote to shared memory.
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status,
                                         bool cluster = false) {
  const bool got = cluster ? mbar_wait_cluster(bar, parity, abort, status) : mbar_wait(bar, parity, abort, status);
  return __all_sync(0xffffffffu, got);
}

// Staging of the outputs.  fp32: each epilogue warp stages 32 i x 32 j (rows of
// 128 bytes).  16-bit: two warps of neighbouring quarters stage 64 i x 64 j
// together, so that rows are 128 bytes there too: the TMA unit, which also
// brings the operands, spends as long on a row of 64 bytes as on one of 128.
// The buffer is free again once the store that used it last has read it.
struct OutStage {
  uint8_t* buf;
  uint64_t* bar;          // 16-bit: the two warps' barrier
  uint32_t phase;
  bool issuer;            // this warp hands the buffer to TMA
  volatile int* abort;
  int32_t* status;
  // both warps of a 16-bit buffer; false after a timeout (nothing is left waiting)
  __device__ __forceinline__ bool pair_sync() {
    __syncwarp();
    if (elect_one()) mbar_arrive(bar);
    const bool ok = all_wait(bar, phase, abort, status);
    phase ^= 1u;
    return ok;
  }
};

// Byte offset of 16-byte piece c of row r of the staging: 16-bit buffers carry
// TMA's 128-byte swizzle, which spreads the 8 rows a transposing store writes
// at once over all banks.
template <int ELEM> __device__ __forceinline__ int box_piece(int r, int c) {
  return r * 128 + (ELEM == 4 ? c : c ^ (r & 7)) * 16;
}

// The staged rows to out rows row.. at column j; `left` of them count (a
// multiple of 32 except at the end of i).  Whole boxes go by TMA, which clips
// at the edges of the output matrix (wgrad: of the expert's matrix); a
// group's last rows are stored by the threads, since a box would write the
// next group's rows.  The staged values are visible to TMA and to the threads.
template <int FORM, int ELEM>
__device__ __forceinline__ void flush(const ProductParams& p, const OutStage& os, int j, int row, int depth,
                                      int left, int lane) {
  constexpr int ROWS = ELEM == 4 ? 32 : 64;
  int done = 0;                                                        // rows that TMA takes
  if (left >= ROWS || (FORM == kWgrad && left > ROWS - 32)) {
    done = ROWS;
    if (os.issuer && elect_one()) {
      if (FORM == kWgrad && ELEM == 4 && p.accumulate) tma_add_3d(&p.tmOut, os.buf, j, row, depth);
      else tma_store_3d(&p.tmOut, os.buf, j, row, depth);
      bulk_commit_group();
    }
  } else if (ELEM == 2 && (FORM == kWgrad || left >= 32)) {
    done = 32;
    if (os.issuer && elect_one()) {
      tma_store_3d(&p.tmOut32, os.buf, j, row, depth);
      bulk_commit_group();
    }
  }
  if (FORM != kWgrad && done < left && done < ROWS) {
    // 8 pieces of 16 bytes a row; two warps take every other run of 32
    const int first = ELEM == 4 || os.issuer ? 0 : 32, step = ELEM == 4 ? 32 : 64;
#pragma unroll 1
    for (int x = done * 8 + first + lane; x < left * 8; x += step) {
      const int r = x >> 3, c = x & 7, jj = j + c * (16 / ELEM);
      if (jj < p.n_j)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) +
                                  (static_cast<int64_t>(row + r) * p.n_j + jj) * ELEM) =
            *reinterpret_cast<const uint4*>(os.buf + box_piece<ELEM>(r, c));
    }
  }
  __syncwarp();
}

template <int OUT> struct Elem {
  using type = float;
  static __device__ __forceinline__ float from(float v) { return v; }
};
template <> struct Elem<MOE_ELEM_BF16> {
  using type = __nv_bfloat16;
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<MOE_ELEM_F16> {
  using type = __half;
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
};

template <int FORM> struct Majors {
  static constexpr bool M_MN = FORM != kForward;   // M side MN-major (j contiguous)
  static constexpr bool N_MN = FORM == kWgrad;     // N side MN-major (i contiguous)
};

// SPLIT: tiles in pieces along r (build_split_tables), which are stored to their
// slots as fp32; whole tiles go to the output as without it.
template <int FORM, int OUT, bool SPLIT>
__global__ void __launch_bounds__(num_threads(FORM), 1)
    grouped_matmul_kernel(const __grid_constant__ ProductParams p) {
  constexpr bool M_MN = Majors<FORM>::M_MN, N_MN = Majors<FORM>::N_MN;
  constexpr bool F32 = OUT == MOE_ELEM_F32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int stages = p.stages;
  uint8_t* ring_end = smem + stages * STAGE_BYTES;
  TileInfo* s_tq = reinterpret_cast<TileInfo*>(ring_end + EPI_WARPS * OUT_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(s_tq + TQ);
  uint64_t* empty = full + STAGES;
  uint64_t* tail = empty + STAGES;       // wgrad: a partial block's loads of this CTA
  uint64_t* tfull = tail + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* tq = drain + 1;              // a tile is in the queue; its readers have it
  uint64_t* tqe = tq + TQ;
  uint64_t* pair = tqe + TQ;             // 16-bit staging: its two warps
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + Smem::kNumBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 2);
  int* s_off = reinterpret_cast<int*>(s_tmem + 4);
  int* s_tile = s_off + (p.E + 1);
  int* s_slot = s_tile + (p.E + 1);      // split products
  int* s_piece = s_bad + 1;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // warp-uniform
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x >> 1);
  const int units = static_cast<int>(gridDim.x >> 1);

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < STAGES; ++i) {
        // one arrival with the expected bytes and, for wgrad, a second one: a
        // partial block has one from each CTA's FIX_WARP instead
        mbar_init(&full[i], FORM == kWgrad ? 2 : 1);
        mbar_init(&empty[i], 1);
        mbar_init(&tail[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&tfull[i], 1);
        mbar_init(&tempty[i], 2 * EPI_WARPS);   // the epilogue warps of both CTAs
      }
      mbar_init(drain, 1);
      for (int i = 0; i < 4; ++i) mbar_init(&pair[i], 2);
      for (int i = 0; i < TQ; ++i) {
        mbar_init(&tq[i], 1);
        // the producer and the epilogue warps; rank 0's issuer; wgrad's FIX_WARP
        mbar_init(&tqe[i], 1 + EPI_WARPS + (leader ? 1 : 0) + (FORM == kWgrad ? 1 : 0));
      }
      *s_abort = 0;
      *s_bad = 0;
      fence_mbar_init();
      fence_proxy_async_smem();
      prefetch_tmap(&p.tmM);
      prefetch_tmap(&p.tmN[0]);
    }
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc_pair(s_tmem, TMEM_COLS);
    tmem_relinquish_pair();
  }
  __syncthreads();                       // *s_bad = 0 before warp 2 may set it
  pdl_wait();
  if (warp == 2) {
    if (SPLIT) {
      build_split_tables<FORM, false>(p, s_off, s_tile, s_slot, s_piece, s_bad);
      if (blockIdx.x == 0 && lane == 0) *p.cut = s_slot[p.E];
    } else {
      build_tables<FORM>(p, s_off, s_tile, s_bad);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                        // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();

  const uint32_t tmem_base = *s_tmem;
  const int total = s_tile[p.E];
  if (threadIdx.x == 0 && *s_bad) record_status(p.status, DEV_BAD_ROW);

  // The tile sequence of this pair: tiles unit, unit + units, ...  A warp of
  // each CTA works them out ahead of the others (a search and a few divisions
  // that would otherwise sit between two tiles' loads and MMAs) and queues
  // them: tile seq in slot seq % TQ, tq[slot] completes when it is there,
  // tqe[slot] when every reader has it.
  auto take = [&](int seq, TileInfo& t) {
    const int slot = seq % TQ;
    if (!all_wait(&tq[slot], (seq / TQ) & 1, s_abort, p.status)) return false;
    t = s_tq[slot];
    __syncwarp();
    if (elect_one()) mbar_arrive(&tqe[slot]);
    return t.blocks >= 0;
  };

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    int stage = 0;
    uint32_t phase = 0;
    uint32_t used = 0, last = 0;               // stages loaded, parity of their last load
    uint32_t tails = 0, tail_par = 0;          // the same for tail[]
    bool ok = true;
    TileInfo t;
    for (int seq = 0; ok && take(seq, t); ++seq) {
      const int j = t.j0 + rank * 128;
      const int half = t.mma_n >> 1;                     // i rows of this CTA
      const int i = t.i0 + rank * half;
      const int n_boxes = N_MN ? (half + 63) >> 6 : 0;
      const uint32_t bytes = SIDE_BYTES + (N_MN ? n_boxes * 8192 : half * (BK * 2));
      // an expert without rows (wgrad) passes one stage on without loads
      if (FORM == kWgrad && t.blocks == 0) {
        if (!all_wait(&empty[stage], phase ^ 1u, s_abort, p.status)) break;
        if (elect_one()) mbar_arrive_cluster_light(mapa_shared(&full[stage], 0));   // both CTAs: 2 arrivals
        __syncwarp();
        used &= ~(1u << stage);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
        continue;
      }
      for (int b = 0; b < t.blocks; ++b) {
        if (!all_wait(&empty[stage], phase ^ 1u, s_abort, p.status)) { ok = false; break; }
        uint8_t* m_dst = smem + stage * STAGE_BYTES;
        uint8_t* n_dst = m_dst + SIDE_BYTES;
        const int r = (SPLIT && FORM != kWgrad ? t.rows + b : b) * BK;
        // wgrad: a last block past the group's rows completes on this CTA's own barrier
        const bool partial = FORM == kWgrad && r + BK > t.rows;
        if (elect_one()) {
          uint32_t bar;
          if (partial) {
            mbar_arrive_expect_tx(&tail[stage], bytes);
            bar = mapa_shared(&tail[stage], static_cast<uint32_t>(rank));
          } else {
            if (leader) {
              mbar_arrive_expect_tx(&full[stage], 2 * bytes);
              if (FORM == kWgrad) mbar_arrive(&full[stage]);
            }
            bar = mapa_shared(&full[stage], 0);
          }
          if (!M_MN) {
            tma_load_3d_pair(m_dst, &p.tmM, bar, r, j, group_of<SPLIT>(t));
          } else if (FORM == kDgrad) {
            tma_load_3d_pair(m_dst, &p.tmM, bar, j, r, group_of<SPLIT>(t));
            tma_load_3d_pair(m_dst + 8192, &p.tmM, bar, j + 64, r, group_of<SPLIT>(t));
          } else {
            tma_load_2d_pair(m_dst, &p.tmM, bar, j, t.row0 + r);
            tma_load_2d_pair(m_dst + 8192, &p.tmM, bar, j + 64, t.row0 + r);
          }
          if (N_MN) {
            for (int x = 0; x < n_boxes; ++x)
              tma_load_2d_pair(n_dst + x * 8192, &p.tmN[0], bar, i + 64 * x, t.row0 + r);
          } else {
            // half (a multiple of 16) as boxes of 128, 64, 32 and 16 rows
            int at = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int h = 128 >> x;
              if (half & h) {
                tma_load_2d_pair(n_dst + at * (BK * 2), &p.tmN[x], bar, r, t.row0 + i + at);
                at += h;
              }
            }
          }
        }
        __syncwarp();
        used = partial ? used & ~(1u << stage) : used | 1u << stage;
        last = (last & ~(1u << stage)) | (phase << stage);
        if (partial) {
          tails |= 1u << stage;
          tail_par ^= 1u << stage;                       // set = parity 0 completed last
        }
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
    }
    pdl_trigger();
    // Wait (bounded) until the last load issued on every stage has landed,
    // so that no copy still writes shared memory when the block exits.
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      for (int s = 0; s < STAGES; ++s) {
        const bool on_full = leader && ((used >> s) & 1u);
        const bool on_tail = (tails >> s) & 1u;
        while ((on_full && !mbar_try_wait(&full[s], (last >> s) & 1u)) ||
               (on_tail && !mbar_try_wait(&tail[s], ((tail_par >> s) & 1u) ^ 1u))) {
          if (globaltimer_ns() - t0 > kWaitLimitNs) { record_status(p.status, DEV_WAIT_TIMEOUT); break; }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer (rank 0)
    if (leader) {
      const uint32_t idesc_base = p.fmt | (1u << 4) | (M_MN ? 1u << 15 : 0u) | (N_MN ? 1u << 16 : 0u) |
                                  (static_cast<uint32_t>(TM >> 4) << 24);
      // one K=16 step: 32 bytes along a K-major row, 16 rows of an MN-major box
      constexpr uint64_t m_step = M_MN ? 2048 >> 4 : 32 >> 4, n_step = N_MN ? 2048 >> 4 : 32 >> 4;
      constexpr uint64_t next_stage = STAGE_BYTES >> 4;
      const uint32_t s0 = smem_u32(smem);
      const uint64_t mdesc0 = M_MN ? smem_desc_mnmajor_sw128(s0) : smem_desc_kmajor_sw128(s0);
      const uint64_t ndesc0 = N_MN ? smem_desc_mnmajor_sw128(s0 + SIDE_BYTES) : smem_desc_kmajor_sw128(s0 + SIDE_BYTES);
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;                                          // chains so far
      bool ok = true;
      TileInfo t;
      for (int seq = 0; ok && take(seq, t); ++seq) {
        t.blocks = __shfl_sync(0xffffffffu, t.blocks, 0);   // uniform registers again
        t.rows = __shfl_sync(0xffffffffu, t.rows, 0);
        t.mma_n = __shfl_sync(0xffffffffu, t.mma_n, 0);
        const uint32_t idesc = idesc_base | (static_cast<uint32_t>(t.mma_n >> 3) << 17);
        // an expert without rows: one stage without MMAs
        const int blocks = FORM == kWgrad ? max(t.blocks, 1) : t.blocks;
        for (int b0 = 0; b0 < blocks && ok; b0 += kChain, ++it) {
          const int acc = it & 1;
          const int b1 = min(blocks, b0 + kChain);
          if (!all_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, s_abort, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * TN);
          for (int b = b0; b < b1; ++b) {
            // a partial block (wgrad) has been mended by threads of both CTAs
            const bool partial = FORM == kWgrad && (b + 1) * BK > t.rows;
            if (!all_wait(&full[stage], phase, s_abort, p.status, partial)) { ok = false; break; }
            tc_fence_after();
            const uint64_t mdesc = mdesc0 + stage * next_stage, ndesc = ndesc0 + stage * next_stage;
            const int steps = partial ? (t.rows - b * BK + 15) >> 4 : BK / 16;
            if (elect_one()) {
#pragma unroll
              for (int s = 0; s < BK / 16; ++s)
                if (FORM != kWgrad || s < steps)
                  mma_bf16_ss_pair(d_tmem, mdesc + s * m_step, ndesc + s * n_step, idesc,
                                   b > b0 || s > 0 ? 1u : 0u);
              mma_commit_pair(&empty[stage], 0x3);         // frees the stage in both CTAs
              if (b + 1 == b1) mma_commit_pair(&tfull[acc], 0x3);
            }
            __syncwarp();
            if (++stage == stages) { stage = 0; phase ^= 1u; }
          }
        }
      }
      // every MMA issued must be complete before tensor memory is freed
      if (elect_one()) {
        mma_commit_pair(drain, 0x1);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0)) {
          if (globaltimer_ns() - t0 > kWaitLimitNs) { record_status(p.status, DEV_WAIT_TIMEOUT); break; }
        }
      }
    }
    __syncwarp();
  } else if (warp == SCHED_WARP) {
    // ------------------------------------------------------------- scheduler
    for (int seq = 0;; ++seq) {
      const int slot = seq % TQ;
      const int64_t tile = unit + static_cast<int64_t>(seq) * units;
      TileInfo t;
      t.blocks = -1;
      if (tile < total) t = tile_info<FORM, SPLIT>(static_cast<int>(tile), p, s_off, s_tile, s_slot, *s_piece);
      if (!all_wait(&tqe[slot], ((seq / TQ) & 1) ^ 1u, s_abort, p.status)) break;
      if (elect_one()) {
        s_tq[slot] = t;
        mbar_arrive(&tq[slot]);
      }
      __syncwarp();
      if (t.blocks < 0) break;
    }
  } else if (FORM == kWgrad && warp == FIX_WARP) {
    // -------------------------- wgrad: the partial last block of a group's rows
    int stage = 0;
    uint32_t tail_par = 0;
    TileInfo t;
    for (int seq = 0; take(seq, t); ++seq) {
      if (t.blocks == 0) {
        stage = (stage + 1) % stages;
        continue;
      }
      stage = (stage + t.blocks - 1) % stages;             // the last block's stage
      const int valid = t.rows - (t.blocks - 1) * BK;
      if (valid < BK) {
        // this CTA's loads have landed (every lane waits, so that its stores
        // follow them): zero the rows past the group up to the next multiple
        // of 16, in both operands
        if (!all_wait(&tail[stage], (tail_par >> stage) & 1u, s_abort, p.status)) break;
        tail_par ^= 1u << stage;
        uint8_t* base = smem + stage * STAGE_BYTES + valid * 128;
        const int count = (((valid + 15) & ~15) - valid) * 8;       // 16-byte pieces a box
        const int boxes = 2 + (((t.mma_n >> 1) + 63) >> 6);
        for (int box = 0; box < boxes; ++box)                       // M side's two, then N side's
          for (int x = lane; x < count; x += 32)
            *reinterpret_cast<uint4*>(base + box * 8192 + x * 16) = make_uint4(0, 0, 0, 0);
        // The MMA that reads these zeros is issued by rank 0: each lane's stores
        // are made visible to the async proxy, gathered by the warp's barrier, and
        // released at cluster scope by the arrival that the issuer acquires.  The
        // release covers shared memory alone: one over all memory waits for other
        // warps' outputs too (24576 rows of 64 experts: 254 us against 230).
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_smem(mapa_shared(&full[stage], 0));
      }
      stage = (stage + 1) % stages;
    }
  } else if (warp >= 2 && warp < 2 + EPI_WARPS) {
    // -------------------------------------------------------------- epilogue
    // Warp w stores the lanes of quarter w % 4 (32 j) and every other run of
    // 64 (fp32: 32) columns (i).
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const int sharing = part * 2 + (quarter >> 1);         // 16-bit: this warp's buffer
    OutStage os{ring_end + (F32 ? (warp - 2) * OUT_BYTES : sharing * 2 * OUT_BYTES), &pair[sharing], 0,
                F32 || (quarter & 1) == 0, s_abort, p.status};
    // transposing stores: lane 8m + r gives row r of an 8-row group, piece m
    const uint32_t st_addr =
        smem_u32(os.buf) + static_cast<uint32_t>(box_piece<2>(lane & 7, (quarter & 1) * 4 + (lane >> 3)));
    int it = 0;
    bool ok = true;
    TileInfo t;
    for (int seq = 0; ok && take(seq, t); ++seq) {
      const int j = t.j0 + rank * 128 + quarter * 32;
      const int row = FORM == kWgrad ? t.i0 : t.row0 + t.i0;   // output row of column 0
      const int depth = FORM == kWgrad ? group_of<SPLIT>(t) : 0;
      const int slot = SPLIT ? (t.e >> kGroupBits) - 1 : -1;
      const int blocks = FORM == kWgrad ? max(t.blocks, 1) : t.blocks;
      // the tile's chains are added in registers, in order
      auto wait_chain = [&] {
        if (!warp_wait(&tfull[it & 1], (it >> 1) & 1, s_abort, p.status)) return false;
        tc_fence_after();
        return true;
      };
      auto release_chain = [&] {                           // to the issuer's barrier
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_light(mapa_shared(&tempty[it & 1], 0));
      };
      if (F32 || (SPLIT && slot >= 0)) {
        // fp32, and pieces: a lane holds a row of the accumulator
        float sum[4][32];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[x][i] = 0.0f;   // also what an expert without rows gets
        for (int b = 0; b < blocks; b += kChain, ++it) {
          if (!wait_chain()) { ok = false; break; }
          const uint32_t src = t_lane + static_cast<uint32_t>((it & 1) * TN);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int c = (2 * x + part) * 32;
            if (c < t.ni && t.blocks > 0) {                // warp-uniform
              uint32_t v[32];
              tmem_ld_32x32b_x32(src + static_cast<uint32_t>(c), v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) sum[x][i] += __uint_as_float(v[i]);
            }
          }
          release_chain();
        }
        if (!ok) break;
        uint8_t* buf = os.buf;
        if (!F32) {
          // each warp in its half of the two warps' buffer, which the issuer's
          // last store may still be reading
          if (elect_one()) bulk_wait_group_read0();
          if (!os.pair_sync()) { ok = false; break; }
          buf += (quarter & 1) * OUT_BYTES;
        }
        if (j < p.n_j) {                                   // warp-uniform
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int c = (2 * x + part) * 32;
            if (c < t.ni) {
              if (elect_one()) bulk_wait_group_read0();
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 32; ++i) *reinterpret_cast<float*>(buf + i * 128 + lane * 4) = sum[x][i];
              fence_proxy_async_smem();
              __syncwarp();
              if (SPLIT && slot >= 0) {                    // a whole box: the slot is this piece's alone
                if (elect_one()) {
                  tma_store_3d(&p.tmParts, buf, j - t.j0, slot * p.slot_i + c, 0);
                  bulk_commit_group();
                }
                __syncwarp();
              } else if constexpr (F32) {
                flush<FORM, 4>(p, os, j, row + c, depth, t.ni - c, lane);
              }
            }
          }
        }
      } else {
        // 64 columns at a time: 8 x 8 fragments, rounded in pairs and stored
        // transposed
        float sum[2][64];                                  // [64 columns][lane half][column half][16]
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 64; ++i) sum[x][i] = 0.0f;
        for (int b = 0; b < blocks; b += kChain, ++it) {
          if (!wait_chain()) { ok = false; break; }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int c = part * 64 + (y >> 1) * 128 + (y & 1) * 32;
            if (c < t.ni && t.blocks > 0) {                // warp-uniform
              const uint32_t src = t_lane + static_cast<uint32_t>((it & 1) * TN + c);
              uint32_t v[32];
              tmem_ld_16x256b_x4(src, v);
              tmem_ld_16x256b_x4(src + (16u << 16), v + 16);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                sum[y >> 1][(i >> 4) * 32 + (y & 1) * 16 + (i & 15)] += __uint_as_float(v[i]);
            }
          }
          release_chain();
        }
        if (!ok) break;
        const int j_box = j & ~63;                         // both warps' 64 columns
        if (j_box < p.n_j) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int c = part * 64 + x * 128;
            if (c >= t.ni) break;
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float lo = sum[x][2 * i], hi = sum[x][2 * i + 1];
              if (OUT == MOE_ELEM_F16) {
                const __half2 h = __floats2half2_rn(lo, hi);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
              } else {
                w[i] = pack_bf16x2(lo, hi);
              }
            }
            if ((SPLIT || os.issuer) && elect_one()) bulk_wait_group_read0();   // split: a piece's boxes too
            if (!os.pair_sync()) { ok = false; break; }
            // w[16 h16 + 8 half + 2 n + h8]: j 16 h16 + 8 h8 .., i 32 half + 8 n ..
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int n = 0; n < 4; ++n)
                stmatrix_x4_trans(st_addr + half * 4096 + n * 1024, w[8 * half + 2 * n], w[8 * half + 2 * n + 1],
                                  w[16 + 8 * half + 2 * n], w[16 + 8 * half + 2 * n + 1]);
            fence_proxy_async_smem();
            if (!os.pair_sync()) { ok = false; break; }
            flush<FORM, 2>(p, os, j_box, row + c, depth, t.ni - c, lane);
          }
        }
      }
    }
    // the warp's stores complete before the block (and its shared memory) goes
    if (elect_one()) bulk_wait_group0();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                        // no MMA or signal of the pair is still in flight
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// The pieces of a split product's tiles, added in order and rounded once.  A
// step is 256 j by kJoinRows i, or by four times as many where there are steps
// enough for every block: a thread takes four j, of V i, with 16 loads in flight.
struct JoinParams : Shape {
  const float* parts;
  void* out;
};

template <int FORM, int OUT, int V>
__device__ __forceinline__ void join_step(const JoinParams& p, int step, int steps, const int* s_off,
                                          const int* s_tile, const int* s_slot) {
  using O = typename Elem<OUT>::type;
  constexpr int U = 16 / V;
  const int tile = step / steps, i0 = (step - tile * steps) * (kJoinRows * V) + (threadIdx.x >> 6);
  const int e = find_group(tile, p.E, s_tile);
  const int n_i = FORM == kWgrad ? p.n_i : s_off[e + 1] - s_off[e];
  const int it = tiles_over(n_i, TN), jt = tiles_over(p.n_j, TM);
  const int local = tile - s_tile[e];
  int i, j;
  tile_at(local, it, jt, i, j);
  const int h = even_height(n_i), jj = (threadIdx.x & 63) * 4;
  const int ni = min(h, n_i - i * h);
  if (i0 >= ni || j * TM + jj >= p.n_j) return;            // n_j: a multiple of 8
  const int pieces = (s_slot[e + 1] - s_slot[e]) / (it * jt);
  const int64_t slot_size = static_cast<int64_t>(p.slot_i) * p.slot_j;
  const int64_t stride = it * jt * slot_size;
  const float* src = p.parts + (s_slot[e] + local) * slot_size + static_cast<int64_t>(i0) * p.slot_j + jj;
  O* out = static_cast<O*>(p.out) +
           ((FORM == kWgrad ? static_cast<int64_t>(e) * p.n_i : static_cast<int64_t>(s_off[e])) + i * h + i0) * p.n_j +
           j * TM + jj;
  // an old weight gradient, loaded ahead and added last: pieces added to it one
  // by one would each be rounded at its size
  float4 sum[V], old[V];
#pragma unroll
  for (int r = 0; r < V; ++r) {
    sum[r] = old[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (OUT == MOE_ELEM_F32)
      if (FORM == kWgrad && p.accumulate && i0 + r * kJoinRows < ni)
        old[r] = *reinterpret_cast<const float4*>(out + static_cast<int64_t>(r * kJoinRows) * p.n_j);
  }
  for (int q = 0; q < pieces; q += U) {
    float4 v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < V; ++r)
        v[u][r] = q + u < pieces && i0 + r * kJoinRows < ni
                      ? *reinterpret_cast<const float4*>(src + (q + u) * stride + r * kJoinRows * p.slot_j)
                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < V; ++r) {
        sum[r].x += v[u][r].x;
        sum[r].y += v[u][r].y;
        sum[r].z += v[u][r].z;
        sum[r].w += v[u][r].w;
      }
  }
#pragma unroll
  for (int r = 0; r < V; ++r) {
    if (i0 + r * kJoinRows >= ni) continue;
    O* dst = out + static_cast<int64_t>(r * kJoinRows) * p.n_j;
    if constexpr (OUT == MOE_ELEM_F32) {
      *reinterpret_cast<float4*>(dst) =
          make_float4(old[r].x + sum[r].x, old[r].y + sum[r].y, old[r].z + sum[r].z, old[r].w + sum[r].w);
    } else {
      const O w[4] = {Elem<OUT>::from(sum[r].x), Elem<OUT>::from(sum[r].y), Elem<OUT>::from(sum[r].z),
                      Elem<OUT>::from(sum[r].w)};
      *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(w);
    }
  }
}

template <int FORM, int OUT>
__global__ void __launch_bounds__(256, 2) join_pieces_kernel(const JoinParams p) {
  extern __shared__ int s_tables[];
  __shared__ int s_piece, s_bad;
  int* s_off = s_tables;
  int* s_tile = s_off + (p.E + 1);
  int* s_slot = s_tile + (p.E + 1);
  pdl_wait();
  pdl_trigger();
  if (*p.cut == 0) return;                                 // no tile in pieces
  if (threadIdx.x < 32) build_split_tables<FORM, true>(p, s_off, s_tile, s_slot, &s_piece, &s_bad);
  __syncthreads();
  const int tiles = s_tile[p.E];
  const int wide = (p.slot_i + 4 * kJoinRows - 1) / (4 * kJoinRows), steps = (p.slot_i + kJoinRows - 1) / kJoinRows;
  if (tiles * steps > static_cast<int>(gridDim.x)) {
    for (int x = blockIdx.x; x < tiles * wide; x += gridDim.x)
      join_step<FORM, OUT, 4>(p, x, wide, s_off, s_tile, s_slot);
  } else if (static_cast<int>(blockIdx.x) < tiles * steps) {
    join_step<FORM, OUT, 1>(p, blockIdx.x, steps, s_off, s_tile, s_slot);
  }
}

// ----------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// Tensor of `depth` matrices [rows, cols] (depth 0: one, as a 2-D map), boxes
// of box_cols x box_rows, swizzled as told.
bool encode(CUtensorMap* m, const void* base, int elem, int64_t cols, int64_t rows, int depth, int box_cols,
            int box_rows, CUtensorMapSwizzle swizzle) {
  auto fn = encoder();
  if (fn == nullptr) return false;
  const cuuint64_t size = elem == MOE_ELEM_F32 ? 4 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(depth)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * size,
                           static_cast<cuuint64_t>(cols) * size * static_cast<cuuint64_t>(rows)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType type = elem == MOE_ELEM_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : elem == MOE_ELEM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(m, type, depth > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FORM, int OUT, bool SPLIT>
cudaError_t launch_form(ProductParams p, int64_t max_tiles, int num_sms, cudaStream_t stream) {
  p.stages = Smem::bytes(p.E, STAGES, SPLIT) <= kMaxSmem ? STAGES : STAGES - 1;
  const int smem = Smem::bytes(p.E, p.stages, SPLIT);
  static std::atomic<int> configured[64];
  int dev = 0;
  cudaGetDevice(&dev);
  const bool cached = dev >= 0 && dev < 64;
  if (!cached || configured[dev].load(std::memory_order_relaxed) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(grouped_matmul_kernel<FORM, OUT, SPLIT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    if (cached) configured[dev].store(1, std::memory_order_relaxed);
  }
  int64_t units = num_sms / 2;
  if (SPLIT) units = std::min<int64_t>(units, kSplitUnits);
  else if (max_tiles < units) units = max_tiles > 0 ? max_tiles : 1;
  p.units = static_cast<int>(units);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * units), 1, 1);
  cfg.blockDim = dim3(num_threads(FORM), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_matmul_kernel<FORM, OUT, SPLIT>, p);
}

template <int FORM, int OUT>
cudaError_t launch_split(const ProductParams& p, float* parts, int num_sms, cudaStream_t stream) {
  const cudaError_t e = launch_form<FORM, OUT, true>(p, 0, num_sms, stream);
  if (e != cudaSuccess) return e;
  JoinParams q{};
  static_cast<Shape&>(q) = p;
  q.units = std::min(num_sms / 2, kSplitUnits);
  q.parts = parts;
  q.out = p.out;
  const size_t smem = sizeof(int) * 3 * (static_cast<size_t>(p.E) + 1);
  return launch_chained(join_pieces_kernel<FORM, OUT>, dim3(static_cast<unsigned>(2 * num_sms)), dim3(256), smem,
                        stream, q);
}

template <int OUT>
cudaError_t launch_out(int form, const ProductParams& p, float* parts, int64_t max_tiles, int num_sms,
                       cudaStream_t stream) {
  if (parts != nullptr)
    return form == kForward ? launch_split<kForward, OUT>(p, parts, num_sms, stream)
           : form == kDgrad ? launch_split<kDgrad, OUT>(p, parts, num_sms, stream)
                            : launch_split<kWgrad, OUT>(p, parts, num_sms, stream);
  return form == kForward ? launch_form<kForward, OUT, false>(p, max_tiles, num_sms, stream)
         : form == kDgrad ? launch_form<kDgrad, OUT, false>(p, max_tiles, num_sms, stream)
                          : launch_form<kWgrad, OUT, false>(p, max_tiles, num_sms, stream);
}

// Slots of a product whose tiles may be cut along r.  Cutting needs a second
// launch, 2 us where nothing is cut and 4 to 6 us where something is; 64 of r
// take a pair 0.27 us.  So it is for
//   forward, dgrad  as many groups as rows allow leave half of the pairs without
//                   a tile, and r has at least 48 blocks (256 rows, n = 2560 to
//                   256 columns 22 us cut, 24 whole; n = 2048 21 both ways)
//   wgrad           groups of even length leave half of the pairs without a tile
//                   and have 48 blocks each (4096 rows, 256 x 256: 16 us cut, 24
//                   whole; 3136 rows 16 and 20), or kSkewedRows rows, few tiles a
//                   group, and possibly most rows in one group (16 groups of 32768
//                   rows, 512 x 512: even 23 us cut, 21 whole; longest 9592 rows 41
//                   and 53.  64 of 65536: even 41 and 43, all rows in one 54 and 303)
struct Slots { int count, i, j; };
Slots split_slots(int form, int64_t rows, int E, int n, int k) {
  constexpr int64_t kMinBlocks = 6 * kMinPiece;
  const int n_j = form == kForward ? n : k;
  const int64_t jt = tiles_over(n_j, TM);
  bool cut;
  if (form == kWgrad) {
    const int64_t tiles = tiles_over(n, TN) * jt;
    cut = (2 * tiles * E <= kSplitUnits && ceil_div(rows, BK) >= kMinBlocks * E) ||
          (4 * tiles <= kSplitUnits && rows >= kSkewedRows);
  } else {
    const int64_t tiles = std::max<int64_t>(std::min<int64_t>(rows, E), ceil_div(rows, TN)) * jt;
    cut = rows > 0 && 2 * tiles <= kSplitUnits && tiles_over(form == kForward ? k : n, BK) >= kMinBlocks;
  }
  if (!cut) return {0, 0, 0};
  const int64_t i_side = form == kWgrad ? n : std::min<int64_t>(rows, TN);
  return {2 * kSplitUnits, even_height(static_cast<int>(i_side)), std::min<int>(TM, (n_j + 31) & ~31)};
}
size_t slots_bytes(const Slots& s) {
  return sizeof(float) * static_cast<size_t>(s.count) * static_cast<size_t>(s.i) * static_cast<size_t>(s.j);
}

}  // namespace

bool grouped_matmul_sm100_takes(const GroupedProduct& g) {
  return g.dtype != MOE_ELEM_F32 && g.n % 8 == 0 && g.k % 8 == 0;
}

size_t grouped_matmul_sm100_parts_bytes(const GroupedProduct& g, int form) {
  return grouped_matmul_sm100_takes(g) ? slots_bytes(split_slots(form, g.rows, g.E, g.n, g.k)) : 0;
}

cudaError_t launch_grouped_matmul_sm100(const GroupedProduct& g, int num_sms, cudaStream_t stream,
                                        bool* map_error) {
  *map_error = false;
  const int f16 = g.dtype == MOE_ELEM_F16;
  ProductParams p{};
  p.offsets = g.offsets;
  p.status = g.status;
  p.out = g.out;
  p.E = g.E;
  p.rows_cap = static_cast<int>(g.rows);
  const bool f32 = g.out_dtype == MOE_ELEM_F32;
  p.accumulate = g.accumulate;
  p.fmt = f16 ? 0u : (1u << 7) | (1u << 10);
  const int64_t rows = g.rows > 0 ? g.rows : 1;   // wgrad of no rows: maps are never read
  const CUtensorMapSwizzle kIn = CU_TENSOR_MAP_SWIZZLE_128B;
  const CUtensorMapSwizzle kOut = f32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok;
  int64_t max_tiles;
  if (g.form == kWgrad) {
    p.n_i = g.n;
    p.n_j = g.k;
    const void* any = g.rows > 0 ? g.q : g.out;
    ok = encode(&p.tmM, any, g.dtype, g.k, rows, 0, BK, BK, kIn) &&
         encode(&p.tmN[0], g.rows > 0 ? g.p : g.out, g.dtype, g.n, rows, 0, BK, BK, kIn) &&
         encode(&p.tmOut, g.out, g.out_dtype, g.k, g.n, g.E, f32 ? 32 : 64, f32 ? 32 : 64, kOut) &&
         encode(&p.tmOut32, g.out, g.out_dtype, g.k, g.n, g.E, f32 ? 32 : 64, 32, kOut);
    p.tmN[1] = p.tmN[2] = p.tmN[3] = p.tmN[0];
    max_tiles = static_cast<int64_t>(g.E) * tiles_over(g.n, TN) * tiles_over(g.k, TM);
  } else {
    const int red = g.form == kForward ? g.k : g.n;
    p.n_j = g.form == kForward ? g.n : g.k;
    p.n_r = red;
    // forward: boxes of 64 k x 128 n; dgrad: 64 k x 64 n (k is j)
    ok = encode(&p.tmM, g.q, g.dtype, g.k, g.n, g.E, BK, g.form == kForward ? 128 : BK, kIn) &&
         encode(&p.tmOut, g.out, g.out_dtype, p.n_j, g.rows, 1, f32 ? 32 : 64, f32 ? 32 : 64, kOut) &&
         encode(&p.tmOut32, g.out, g.out_dtype, p.n_j, g.rows, 1, f32 ? 32 : 64, 32, kOut);
    for (int x = 0; x < 4; ++x)
      ok = ok && encode(&p.tmN[x], g.p, g.dtype, red, rows, 0, BK, 128 >> x, kIn);
    max_tiles = (ceil_div(g.rows, TN) + g.E) * tiles_over(p.n_j, TM);
  }
  const Slots slots = split_slots(g.form, g.rows, g.E, g.n, g.k);
  float* parts = slots.count > 0 ? g.parts : nullptr;
  if (parts != nullptr) {
    p.slot_i = slots.i;
    p.slot_j = slots.j;
    p.cut = g.status + kCutWord;
    ok = ok && encode(&p.tmParts, parts, MOE_ELEM_F32, slots.j, static_cast<int64_t>(slots.count) * slots.i, 1, 32, 32,
                      CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  if (!ok) { *map_error = true; return cudaErrorInvalidValue; }
  return f32                              ? launch_out<MOE_ELEM_F32>(g.form, p, parts, max_tiles, num_sms, stream)
         : g.out_dtype == MOE_ELEM_F16    ? launch_out<MOE_ELEM_F16>(g.form, p, parts, max_tiles, num_sms, stream)
                                          : launch_out<MOE_ELEM_BF16>(g.form, p, parts, max_tiles, num_sms, stream);
}

}  // namespace moe
