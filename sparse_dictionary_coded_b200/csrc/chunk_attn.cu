// Attention of new tokens over paged codes (sdk_chunk_attn, include/sdk.h).
//
// The form for many rows (few rows over short contexts go in one pass,
// chunk_direct.cu, over long ones by atoms, chunk_atoms.cu): the context's vectors
//   K_t = sum_j c_tj D_K[i_tj],  V_t = sum_j c_tj D_V[i_tj]
// are rebuilt once per call as fp16 tiles of 128 tokens in the workspace, and
// softmax(scale q K^T) V is computed over the tiles.
//   chunk_prep_kernel   the plan, the queries as fp16 tiles of packed rows
//   rebuild_kernel      the tiles of keys and values (few tokens and rows: with
//                       the plan and the queries)
//   chunk_attn_kernel   the attention
//   chunk_join_kernel   the sums of blocks that several CTAs shared
#include "chunk_plan.cuh"
#include "tc_ptx.cuh"

namespace sdk {

namespace {

constexpr int kRebThreads = 256;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Most blocks of packed rows the requests' new tokens take (per KV head).
int64_t cap_blocks(int B, int64_t n_tok, int g, int max_q) {
  const int64_t each = ((int64_t)max_q * g + kRows - 1) / kRows * B, all = n_tok * g / kRows + B;
  return each < all ? each : all;
}

// What share c of the work starts with, left for chunk_join_kernel.
struct Cut {
  int64_t u0;          // its first unit
  int64_t lo, hi;      // the units of the block that unit belongs to
  int row0, rows, mb, h;
};

struct ChunkLayout {
  size_t units, cuts, qs, qt, kt, vt, ml, po, total;
};

ChunkLayout chunk_layout(int B, int64_t blocks, int Hkv, int d, int64_t cap_tiles, int ctas,
                         bool whole) {
  ChunkLayout l;
  const size_t tiles = (size_t)cap_tiles * Hkv * kTile * d * 2;
  l.units = up256(sizeof(WsHeader) + ((size_t)B + 1) * sizeof(ReqPlan));
  l.cuts = up256(l.units + ((size_t)blocks + 1) * 8);
  l.qs = up256(l.cuts + (whole ? 0 : (size_t)ctas * sizeof(Cut)));
  l.qt = up256(l.qs + (size_t)blocks * Hkv * kRows * 4);
  l.kt = l.qt + (size_t)blocks * Hkv * kRows * d * 2;
  l.vt = l.kt + tiles;
  l.ml = l.vt + tiles;
  const size_t parts = whole ? 0 : (size_t)2 * ctas * kRows;
  l.po = up256(l.ml + parts * 8);
  l.total = up256(l.po + parts * d * 4);
  return l;
}

}  // namespace

// Byte offset of the 16-byte chunk c8 (dims 8 c8 .. 8 c8 + 7) of token row r
// in a tile image: halves of 64 dims, 128-byte rows, chunks XORed with the
// row (the 128-byte swizzle that both the K-major key operand and the
// MN-major value operand of the tensor cores read).
__device__ __forceinline__ int tile_off(int r, int c8) {
  return (c8 >> 3) * (kTile * 128) + r * 128 + (((c8 & 7) ^ (r & 7)) << 4);
}

// The tiles that the rows of block mb of a request see: first and count.
__device__ __forceinline__ void block_tiles(const ChunkParams& p, const ReqPlan& r, int mb, int* first,
                                            int* count) {
  const int lo_row = mb * kRows, hi_row = min(lo_row + kRows, r.n * p.g) - 1;
  const int lo_pos = r.len - r.n + lo_row / p.g, hi_pos = r.len - r.n + hi_row / p.g;
  const int t1 = p.causal ? min(hi_pos + 1, r.len) : r.len;
  const int t0 = p.window > 0 ? max(0, lo_pos - p.window + 1) : 0;
  *first = *count = 0;
  if (t1 > t0) {
    *first = (t0 - r.lo) / kTile;
    *count = (t1 - r.lo + kTile - 1) / kTile - *first;
  }
}

// Units of work of a block: its tiles, and before them what a block costs
// besides (queries in, outputs out, a pipeline filled and drained: 12000
// cycles against 3000 a tile); a block that sees nothing counts as one, so
// that its rows are written.
constexpr int kBlockCost = 4;
__device__ __forceinline__ int block_units(int tiles) { return tiles > 0 ? tiles + kBlockCost : 1; }

constexpr int kMaxShares = 160;    // shares at most (one per SM; chunk_join_kernel's weights)

// One CTA: the running sum of the blocks' units over all requests, every
// request's first one, and the number of shares: as many as CTAs, but of four
// units at least.
__device__ void plan_blocks(const ChunkParams& p, const int32_t* s_block, int64_t* s_warp) {
  int64_t sum = 0, total;
  const int blocks = s_block[p.B];
  __syncthreads();                     // the plan is written
  for (int m0 = 0; m0 < blocks; m0 += kRebThreads) {
    const int m = m0 + threadIdx.x;
    int64_t n = 0;
    if (m < blocks) {
      const int b = find_first(s_block, p.B, m);
      int at, count;
      const ReqPlan r = p.plan[b];
      // a request that the tiles' capacity refused keeps its blocks' places
      if (r.n > 0) block_tiles(p, r, m - s_block[b], &at, &count);
      n = r.n > 0 ? block_units(count) : 0;
    }
    const int64_t upto = sum + block_scan64(n, s_warp, &total);
    if (m < blocks) p.units[m + 1] = upto;
    sum += total;
  }
  if (threadIdx.x == 0) p.units[0] = 0;
  __syncthreads();
  for (int b = threadIdx.x; b <= p.B; b += kRebThreads) {
    p.plan[b].pair0 = s_block[b];
    p.plan[b].work0 = p.units[s_block[b]] * p.Hkv;
    if (b == p.B) {
      const int64_t shares = (p.units[s_block[b]] * p.Hkv + 3) / 4;
      p.plan[b].npair = (int)(shares < p.ctas ? (shares < 1 ? 1 : shares) : p.ctas);
    }
  }
}

// One CTA, p.parts (at most a block of rows per thread, blocks * Hkv <= ctas):
// cuts every block's tiles into parts of S, S the smallest that leaves no more
// parts than CTAs and not too many to join; p.units: the parts before every block, per KV head.
__device__ void plan_parts(const ChunkParams& p, const int32_t* s_block, int64_t* s_warp) {
  __shared__ int s_tiles[kRebThreads];   // -1: a refused request's
  const int blocks = s_block[p.B], m = threadIdx.x, lane = threadIdx.x & 31;
  __syncthreads();                     // the plan is written
  int tiles = -1;
  if (m < blocks) {
    const int b = find_first(s_block, p.B, m);
    int at;
    const ReqPlan r = p.plan[b];
    if (r.n > 0) block_tiles(p, r, m - s_block[b], &at, &tiles);
  }
  s_tiles[m] = tiles;
  __syncthreads();
  const int room = p.ctas / p.Hkv;
  int S = 1;
  auto parts_of = [&](int t) { return t < 0 ? 0 : max((t + S - 1) / S, 1); };
  auto sum_of = [&](auto f) {
    int v = 0;
    for (int i = lane; i < blocks; i += 32) v += f(s_tiles[i]);
    return __reduce_add_sync(0xffffffffu, v);
  };
  S = max((sum_of([](int t) { return max(t, 0); }) + room - 1) / room, 1);
  // a tile takes 1.6 us, a part of a row 0.35 us when joining: 4.5 S^2 >= tiles
  int most = 0;
  for (int i = lane; i < blocks; i += 32) most = max(most, s_tiles[i]);
  most = __reduce_max_sync(0xffffffffu, most);
  while (9 * (int64_t)S * S < 2 * most) ++S;
  while (sum_of(parts_of) > room) S += (S + 7) / 8;   // (one part a block fits)
  int64_t total;
  const int64_t upto = block_scan64(parts_of(tiles), s_warp, &total);
  if (m < blocks) p.units[m + 1] = upto;
  if (m == 0) p.units[0] = 0;
  for (int b = threadIdx.x; b <= p.B; b += kRebThreads) {
    p.plan[b].pair0 = s_block[b];
    if (b == p.B) {
      p.plan[b].npair = (int)total * p.Hkv;
      p.plan[b].ntiles = S;
    }
  }
}

__device__ __forceinline__ void plan_work(const ChunkParams& p, const int32_t* s_block,
                                          int64_t* s_warp) {
  if (p.parts)
    plan_parts(p, s_block, s_warp);
  else
    plan_blocks(p, s_block, s_warp);
}

constexpr int kPackSteps = 4;

// The query rows as tiles of packed rows (row = token * g + head of the
// group), fp16 scaled by a power of two that puts the row's largest entry
// near 2^15 (exact: 8 significand bits), D / 8 lanes a row, a warp four steps
// of rows at a time.
template <int D>
__device__ __forceinline__ void pack_queries(const ChunkParams& p, const int32_t* s_block,
                                             int cta, int ctas) {
  constexpr int kLanesRow = D / 8, kRowsStep = 32 / kLanesRow, kSteps = kPackSteps;
  const int lane = threadIdx.x & 31, chunk = lane % kLanesRow;
  const uint32_t rows = (uint32_t)(p.n_tok * p.Hq);          // below 2^31
  const uint32_t items = (rows + kRowsStep * kSteps - 1) / (kRowsStep * kSteps);
  const uint32_t warps = (uint32_t)ctas * (kRebThreads / 32);
  for (uint32_t it = (uint32_t)cta * (kRebThreads / 32) + (threadIdx.x >> 5); it < items;
       it += warps) {
    uint4 v[kSteps];
    uint32_t row[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      row[k] = (it * kSteps + k) * kRowsStep + lane / kLanesRow;
      v[k] = row[k] < rows ? __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)row[k] * D) + chunk)
                           : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      uint32_t mx = 0u;                // largest |q| as bf16 bits
#pragma unroll
      for (int u = 0; u < 4; ++u) mx = max(mx, max(x[u] & 0x7FFFu, (x[u] >> 16) & 0x7FFFu));
#pragma unroll
      for (int o = kLanesRow / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (row[k] >= rows) continue;
      float up, up2;
      row_scale(mx, 14, &up, &up2);
      uint32_t y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const __half2 hh = __floats2half2_rn(bf16_lo(x[u]) * up * up2, bf16_hi(x[u]) * up * up2);
        y[u] = *reinterpret_cast<const uint32_t*>(&hh);
      }
      const int tok = (int)(row[k] / (uint32_t)p.Hq), hq = (int)row[k] - tok * p.Hq;
      const int b = find_request(p, tok);
      unsigned err;
      const ReqPlan rq = check_request(p, b, &err);
      if (tok < rq.row0 || tok >= rq.row0 + rq.n) continue;   // a row of no request
      const int h = hq / p.g, r = (tok - rq.row0) * p.g + (hq - h * p.g), rb = r % kRows;
      if (s_block[b] + r / kRows >= s_block[b + 1]) continue;   // refused for want of room
      const int64_t block = (int64_t)(s_block[b] + r / kRows) * p.Hkv + h;
      *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.qt) +
                                (block * 2 + rb / kTile) * (kTile * D * 2) +
                                tile_off(rb % kTile, chunk)) = make_uint4(y[0], y[1], y[2], y[3]);
      if (chunk == 0) p.qscale[block * kRows + rb] = p.scale * 1.44269504f / up / up2;
    }
  }
}

// The plan of the call (CTA 0) and the query tiles.  rebuild_kernel runs
// beside it.
template <int D>
__global__ void __launch_bounds__(kRebThreads) chunk_prep_kernel(ChunkParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_tile0 = sm;                  // [B + 1]
  int32_t* s_block = s_tile0 + p.B + 1;   // [B + 1]
  __shared__ int64_t s_warp[32];
  pdl_launch();
  make_plan<false>(p, blockIdx.x == 0, s_tile0, s_block, s_warp);
  pack_queries<D>(p, s_block, blockIdx.x, gridDim.x);
  if (blockIdx.x == 0) plan_work(p, s_block, s_warp);
}

// The rebuilt tiles.  Every CTA scans the requests' tile counts itself.  D / 8
// lanes rebuild one vector (16-byte pieces of an atom's row), a warp a token's
// key and value (two tokens at head_dim 64), TOK of them one after the other.
// Bound by the gathers of 2 x 16 atom rows (8 KB per token and head at
// head_dim 128) from L2: 2.1 GB at 10.7 TB/s for 32768 tokens of 8 heads, with
// 32 warps an SM and about 8 rows a lane in flight (all 16 take registers that
// leave 16 warps: 15 % slower).  With few tokens it is the chain of loads that
// counts, so there a warp takes one and has all 16 rows in flight, and the
// kernel also does chunk_prep_kernel's work (the plan on a CTA of its own).
template <int D, int TOK>
__global__ void __launch_bounds__(kRebThreads, TOK == 1 ? 2 : 4) rebuild_kernel(ChunkParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_tile0 = sm;              // [B + 1]
  int32_t* s_block = s_tile0 + p.B + 1;
  __shared__ int64_t s_warp[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch();
  make_plan<false>(p, TOK == 1 && blockIdx.x == 0, s_tile0, s_block, s_warp);
  int start = (int)blockIdx.x, stride = (int)gridDim.x;
  if (TOK == 1) {
    if (blockIdx.x == 0) {
      plan_work(p, s_block, s_warp);
      return;
    }
    --start;
    --stride;
    // from the last CTA on: the first ones have most of the items
    pack_queries<D>(p, s_block, stride - 1 - start, stride);
  }

  constexpr int LPR = D / 8;           // lanes per record
  constexpr int TPS = 32 / (2 * LPR);  // tokens a warp rebuilds at a time
  constexpr int WPL = 16 / LPR;        // code words a lane holds
  constexpr int kItemTok = TOK * TPS * (kRebThreads / 32);   // tokens of a work item
  const int rec = lane / LPR, sub = lane % LPR;
  const int kv = rec & 1;
  const uint4* dict = reinterpret_cast<const uint4*>(kv ? p.dv : p.dk);
  char* tiles = reinterpret_cast<char*>(kv ? p.vt : p.kt);
  const int64_t items = (int64_t)s_tile0[p.B] * p.Hkv * (kTile / kItemTok);
  for (int64_t it = start; it < items; it += stride) {
    const int part = (int)(it % (kTile / kItemTok));
    const int th = (int)(it / (kTile / kItemTok)), tile = th / p.Hkv, h = th - tile * p.Hkv;
    const int b = find_first(s_tile0, p.B, tile);
    unsigned err;
    const ReqPlan rq = check_request(p, b, &err);
    const int t_tile = rq.lo + (tile - s_tile0[b]) * kTile;
    const int t_end = rq.n > 0 ? rq.len : 0, t_seen = first_seen(p, rq.len, rq.n);
    char* dst = tiles + ((int64_t)tile * p.Hkv + h) * (kTile * D * 2);
    const int r0 = part * kItemTok + warp * (TOK * TPS) + (rec >> 1);   // row of the tile
#pragma unroll 1
    for (int u = 0; u < TOK; ++u) {
      const int r = r0 + u * TPS, t = t_tile + r;
      if (t - (rec >> 1) >= t_end) {   // the warp's tokens lie behind the context
        // their scores are masked whatever the keys are; values must be finite
        if (kv == 1)
          *reinterpret_cast<uint4*>(dst + tile_off(r, sub)) = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      uint32_t w[WPL];
#pragma unroll
      for (int i = 0; i < WPL; ++i) w[i] = 0u;
      if (t >= t_seen && t < t_end) {   // (tokens before the first seen one are zero)
        const int col = t / p.page_size, off = t - col * p.page_size;
        const int page = p.table[(int64_t)b * p.max_pages + col];
        if (page >= 0 && page < p.n_pages) {
          const uint32_t* src =
              p.pages + ((((int64_t)page * p.Hkv + h) * p.page_size + off) * 2 + kv) * kAtoms;
#pragma unroll
          for (int i = 0; i < WPL; ++i) w[i] = src[sub * WPL + i];
        } else if (sub == 0) {
          record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x76000000u | (uint32_t)b);
        }
      }
      bool bad = false;
      const uint4 y = rebuild_piece<D, TOK == 1>(p, dict, w, rec, sub, &bad);
      if (bad) record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x77000000u | (uint32_t)b);
      *reinterpret_cast<uint4*>(dst + tile_off(r, sub)) = y;
    }
  }
  // done only when chunk_prep_kernel is: the next kernel waits for this one alone
  if (TOK > 1) pdl_wait();
}

// ---------------------------------------------------------------- attention
//
// softmax(scale q K^T) V on the 5th-generation tensor cores.  The rows of a
// KV head's query group are packed (row = token * g + head of the group),
// a CTA takes 256 of them as two MMA tiles of 128 and walks the context's
// rebuilt tiles once with the running maximum and sum:
//   S = Q K^T         tcgen05, both operands from shared memory, fp32 in TMEM
//   P = 2^(S c - m)   one row per thread; written back over S as fp16
//   O = O + P V       tcgen05, P from TMEM, V as the MN-major operand
// While the threads of one tile are in their exponentials, the tensor cores
// work on the other's products.  Warps 0-3 and 4-7 hold the rows of the two
// tiles, warp 8 issues the MMAs, warp 9 the copies (a tile image is
// contiguous: one bulk copy each, into a ring).
// The maximum m is only raised when a tile exceeds it by 2^8 (O then is
// rescaled in TMEM, which is rare); P is 2^7 above its nominal range, so it
// stays below 2^15 and its smallest fp16 step is 2^-31 of the row's largest
// term: N tokens lose less than N 2^-32 of that by it (2^18 tokens 2^-14).
// A CTA takes a block (256 packed rows of a KV head), a part of one, or an
// equal share of all blocks' tiles (chunk_cut says which); a block in several
// parts or shares leaves partial sums that chunk_join_kernel joins.
// 2048 tokens over 32768, 32 heads: 953 us alone, 1120 TFLOP/s (packing and
// rebuilding before it 16 and 201); the tensor pipe is busy two thirds of a
// tile's 3000 cycles, the rest is the chain score - maximum - exponentials - P
// of a row (1800 cycles) that the other tile's products hide in part.  In a
// loop of such calls the card is at its power limit (1000 W at 1.5 to 1.8 GHz):
// the first thirty take 1100 us each, later ones 1240, and fewer idle cycles
// bring less than they seem to.
// Tried: a second warpgroup for each tile (half a row a thread) is bound by
// the exponentials at the same time; half of them on the FMA units instead of
// a quarter is 2 % slower, none 1 %.
namespace {

constexpr int kAThreads = 384;     // a warpgroup for each row tile, one of MMA and copy warps
// registers a thread after the split: 256 x 216 + 128 x 72 = 384 x 168, what
// the block is launched with.  The code is compiled for 168, a row's 128 scores
// among them, and spills 312 bytes a thread at either head size.
constexpr int kRegsLaunch = 168, kRegsRows = 216, kRegsRest = 72;
static_assert(256 * kRegsRows + 128 * kRegsRest == kAThreads * kRegsLaunch, "register split");
constexpr float kPUp = 7.0f;       // log2 of P's offset
constexpr float kSlack = 8.0f;     // log2 of how far a tile may exceed m
constexpr int kPolyOf = 4;         // every 4th pair of exponentials on the FMA units

template <int D>
struct ACfg {
  static constexpr int kTileB = kTile * D * 2;             // one Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kOffQ = kStages * kTileB;
  static constexpr int kOffBar = kOffQ + 2 * kTileB;
  static constexpr int kNumBars = 2 * kStages + 2 + 4 + 2 + 2 + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;       // + alignment slack
  static_assert(kSmem <= 232448, "exceeds the 227 KB shared memory of one sm_100 CTA");
  // D f32, A and B f16; S: both K-major, N = 128; O: B MN-major, N = D
  static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) |
                                      ((uint32_t)(kTile >> 4) << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                      ((uint32_t)(kTile >> 4) << 24);
};

// The MMAs' operands by the low halves of their descriptors (tc::smem_desc,
// tc::smem_desc_mn: address and leading offset; the high half is the same for
// all tiles), so that the one issuing thread spends an addition on each.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) {
  return (addr >> 4) | ((uint32_t)(kTile * 128 >> 4) << 16);
}
// The whole warp runs the issuing loop, so that its values stay in uniform
// registers (which the instruction takes its operands from), and the elected
// lane issues four steps of 16 at a time: with one lane in a branch of its
// own the issue was the bound (this kernel for 2048 tokens over 32768, 32
// heads: 1084 us, so 916 us).
// ss: A and B 16 elements (32 bytes) further along K each step; ts: A 8 TMEM
// columns, B 16 rows of 128 bytes.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 da, db;\n\t.reg .b32 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "mov.b32 a, %1;\n\tmov.b32 b, %2;\n\t"
      "mov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
      "add.u32 a, %1, 2;\n\tadd.u32 b, %2, 2;\n\t"
      "mov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, t;\n\t"
      "add.u32 a, %1, 4;\n\tadd.u32 b, %2, 4;\n\t"
      "mov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, t;\n\t"
      "add.u32 a, %1, 6;\n\tadd.u32 b, %2, 6;\n\t"
      "mov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, t;\n\t"
      "}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 da, db;\n\t.reg .b32 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "mov.b32 a, %1;\n\tmov.b32 b, %2;\n\t"
      "mov.b64 db, {b, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 128;\n\t"
      "mov.b64 db, {b, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, t;\n\t"
      "add.u32 a, %1, 16;\n\tadd.u32 b, %2, 256;\n\t"
      "mov.b64 db, {b, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, t;\n\t"
      "add.u32 a, %1, 24;\n\tadd.u32 b, %2, 384;\n\t"
      "mov.b64 db, {b, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, t;\n\t"
      "}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// 32 lanes x 32 bits, 32 and 16 consecutive columns per thread.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^x of two values, x <= 15, on the FMA units: x = n + f with n the nearest
// integer (left in the low bits by adding 1.5 * 2^23), 2^f by a polynomial of
// degree 3 fitted to the relative error on [-1/2, 1/2] with value 1 at 0
// (at most 2^-13.3, a fifth of the fp16 rounding that follows), n added to
// the exponent.  Below -127 the result is 0; NaN stays NaN: it passes the
// clamp and comes back by the last addition of 0 x.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void ex2_fma(uint64_t x2, float* y0, float* y1) {
  const float kBig = 12582912.0f;
  float a, b;
  unpack2(x2, &a, &b);
  x2 = pack2(max_nan(a, -127.0f), max_nan(b, -127.0f));
  const uint64_t t = add2(x2, pack2(kBig, kBig));
  const uint64_t n = add2(t, pack2(-kBig, -kBig));
  const uint64_t f = fma2(n, pack2(-1.0f, -1.0f), x2);
  uint64_t q = fma2(f, pack2(0.05500885908f, 0.05500885908f), pack2(0.2422110112f, 0.2422110112f));
  q = fma2(q, f, pack2(0.6932829447f, 0.6932829447f));
  q = fma2(q, f, pack2(1.0f, 1.0f));
  float t0, t1, q0, q1;
  unpack2(t, &t0, &t1);
  unpack2(q, &q0, &q1);
  q0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
  q1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
  unpack2(fma2(x2, 0ull, pack2(q0, q1)), y0, y1);
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

}  // namespace

// A bounded wait of a whole warp, all lanes with the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          unsigned long long limit = tc::kWaitNs) {
  if (__all_sync(0xffffffffu, tc::mbar_try(bar, parity))) return true;
  return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, limit));
}

// The last i in [0, n) with at(i) <= v (at rising, at(0) <= v), by a whole
// warp: 32 places a step, so that a few dependent loads find it.
template <typename F>
__device__ __forceinline__ int warp_search(int n, int64_t v, F at) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32, i = lo + lane * step;
    const uint32_t under = __ballot_sync(0xffffffffu, lane * step < len && at(i) <= v);
    const int k = 31 - __clz(under | 1u);
    len = min(step, len - k * step);
    lo += k * step;
  }
  return lo;
}

// A CTA's way through the work: all blocks of all KV heads of all requests in
// that order, cut into equal shares of units.  Only a new request is looked
// up, a block's tiles are computed.
struct Walk {
  int64_t u, end;      // next unit, end of the share
  int b, h, mb;
  int off;             // units of the block before u
  int first, count;    // the block's tiles
  ReqPlan rp;

  // by whole warps
  __device__ __forceinline__ void start(const ChunkParams& p, int64_t from, int64_t to) {
    u = from;
    end = to;
    if (u >= end) return;
    b = warp_search(p.B, u, [&](int i) { return p.plan[i].work0; });
    rp = p.plan[b];
    const int64_t* units = p.units + rp.pair0;
    const int64_t base = units[0], per = units[rp.npair] - base, rel = u - rp.work0;
    h = (int)(rel / per);
    const int64_t at = base + rel - h * per;
    mb = warp_search(rp.npair, at, [&](int i) { return units[i]; });
    off = (int)(at - units[mb]);
    block_tiles(p, rp, mb, &first, &count);
  }
  // block m of the call alone, for KV head hh; false: there is none
  __device__ __forceinline__ bool whole(const ChunkParams& p, int m, int hh) {
    b = warp_search(p.B, m, [&](int i) { return (int64_t)p.plan[i].pair0; });
    rp = p.plan[b];
    h = hh;
    mb = m - rp.pair0;
    off = 0;
    if (mb >= rp.npair) return false;              // refused for want of room
    block_tiles(p, rp, mb, &first, &count);
    u = 0;
    end = units();
    return true;
  }
  // of that block only part k of S tiles
  __device__ __forceinline__ void part(int k, int S) {
    if (count == 0) return;
    const int t0 = k * S, t1 = min(t0 + S, count);
    off = k > 0 ? kBlockCost + t0 : 0;
    end = kBlockCost + t1 - off;
  }
  __device__ __forceinline__ int units() const { return block_units(count); }   // of the block
  // units of the segment that starts at u
  __device__ __forceinline__ int take() const {
    return (int)min((int64_t)(units() - off), end - u);
  }
  // its tiles: `at` the first, of n units
  __device__ __forceinline__ int tiles(int n, int* at) const {
    const int t0 = max(off - kBlockCost, 0), t1 = max(off + n - kBlockCost, 0);
    *at = first + t0;
    return count > 0 ? t1 - t0 : 0;
  }
  __device__ __forceinline__ void next(const ChunkParams& p, int taken) {
    u += taken;
    off = 0;
    if (u >= end) return;
    if (++mb == rp.npair) {
      mb = 0;
      if (++h == p.Hkv) {
        h = 0;
        do ++b;
        while (p.plan[b].npair == 0);
        rp = p.plan[b];
      }
    }
    block_tiles(p, rp, mb, &first, &count);
  }
};

template <int D>
__global__ void __launch_bounds__(kAThreads, 1) chunk_attn_kernel(ChunkParams p) {
  using C = ACfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const int g = p.g;
  pdl_launch();
  pdl_wait();
  int64_t u0 = 0, cut_lo = 0, cut_hi = 0;          // what chunk_join_kernel is told
  Walk walk;
  if (p.whole) {                                   // CTA = block
    // a head's blocks side by side, so that their CTAs read the same tiles at
    // the same time; the longest of a causal call first
    const int blocks = p.plan[p.B].pair0;
    if (blocks == 0) return;
    const int head = (int)blockIdx.x / blocks, m = blocks - 1 - (int)blockIdx.x % blocks;
    if (head >= p.Hkv || !walk.whole(p, m, head)) return;
  } else if (p.parts) {                            // CTA = part of a block
    const int blocks = p.plan[p.B].pair0, S = p.plan[p.B].ntiles, item = (int)blockIdx.x;
    if (item >= p.plan[p.B].npair) return;
    const int m = warp_search(blocks, item, [&](int i) { return p.units[i] * p.Hkv; });
    const int first = (int)p.units[m] * p.Hkv, n = (int)(p.units[m + 1] - p.units[m]);
    const int head = (item - first) / n, k = (item - first) - head * n;
    if (!walk.whole(p, m, head)) return;
    walk.part(k, S);
    u0 = item;                                     // its parts count as units
    cut_lo = item - k;
    cut_hi = cut_lo + n;
  } else {
    const int64_t total = p.plan[p.B].work0;
    const int shares = p.plan[p.B].npair;
    if ((int)blockIdx.x >= shares) return;
    u0 = total * blockIdx.x / shares;
    walk.start(p, u0, total * (blockIdx.x + 1) / shares);
    cut_lo = u0 - walk.off;
    cut_hi = cut_lo + walk.units();
  }
  uint8_t* smem = tc::align_smem_1k(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile uint32_t* s_abort = misc + 0;
  volatile uint32_t* s_tmem = misc + 1;
  const uint32_t s0 = tc::smem_u32(smem);
  auto bar_full = [&](int s) { return tc::smem_u32(&bars[s]); };
  auto bar_empty = [&](int s) { return tc::smem_u32(&bars[C::kStages + s]); };
  auto bar_s = [&](int i) { return tc::smem_u32(&bars[2 * C::kStages + i]); };
  auto bar_p = [&](int i, int half) {
    return tc::smem_u32(&bars[2 * C::kStages + 2 + 2 * i + half]);
  };
  auto bar_q = [&](int i) { return tc::smem_u32(&bars[2 * C::kStages + 6 + i]); };
  auto bar_qfree = [&](int i) { return tc::smem_u32(&bars[2 * C::kStages + 8 + i]); };
  const uint32_t bar_done = tc::smem_u32(&bars[2 * C::kStages + 10]);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *s_abort = 0u;
    for (int s = 0; s < 2 * C::kStages + 2; ++s) tc::mbar_init(tc::smem_u32(&bars[s]), 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(bar_p(i >> 1, i & 1), 4);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar_q(i), 1);
      tc::mbar_init(bar_qfree(i), 4);
    }
    tc::mbar_init(bar_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tc::smem_u32((const void*)s_tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  auto tm_s = [&](int i) { return tmem + (uint32_t)(i * kTile); };          // S, and P over it
  auto tm_o = [&](int i) { return tmem + (uint32_t)(2 * kTile + i * D); };

  // Each role walks the segments by itself; the barriers' phases run on from
  // one segment to the next.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    // the ring's next stage and its parity
    int st = 0;
    uint32_t par = 0;
    auto next_stage = [&]() {
      if (++st == C::kStages) {
        st = 0;
        par ^= 1u;
      }
    };
    Walk w = walk;
    if (warp == 9 && lane == 0) {
      // ----------------------------------------------------------- copies
      const char* kt = reinterpret_cast<const char*>(p.kt);
      const char* vt = reinterpret_cast<const char*>(p.vt);
      bool ok = true;
      uint32_t used = 0u, last = 0u;               // stages written, their latest parity
      uint32_t pqf[2] = {1u, 1u}, qs = 0u;         // parity of bar_qfree, q tiles loaded
      while (ok && w.u < w.end) {
        int at;
        const int n = w.take(), nt = w.tiles(n, &at);
        const int64_t tile0 = w.rp.tile0 + at;
        for (int k = 0; k < 2 * nt && ok; ++k) {
          if (k == 1) {                            // the first keys do not wait for the rows' turn
            const int nact = w.rp.n * g - w.mb * kRows > kTile ? 2 : 1;
            const char* qt = reinterpret_cast<const char*>(p.qt) +
                             ((int64_t)(w.rp.pair0 + w.mb) * p.Hkv + w.h) * 2 * C::kTileB;
            for (int i = 0; i < nact && ok; ++i) {
              ok = tc::mbar_wait(bar_qfree(i), pqf[i], s_abort);
              if (!ok) break;
              pqf[i] ^= 1u;
              tc::mbar_expect_tx(bar_q(i), (uint32_t)C::kTileB);
              bulk_load(s0 + C::kOffQ + i * C::kTileB, qt + i * C::kTileB, (uint32_t)C::kTileB,
                        bar_q(i));
              qs |= 1u << i;
            }
          }
          if (!ok || !tc::mbar_wait(bar_empty(st), par ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          const int64_t tile = (tile0 + (k >> 1)) * p.Hkv + w.h;
          tc::mbar_expect_tx(bar_full(st), (uint32_t)C::kTileB);
          bulk_load(s0 + st * C::kTileB, ((k & 1) ? vt : kt) + tile * C::kTileB,
                    (uint32_t)C::kTileB, bar_full(st));
          used |= 1u << st;
          last = (last & ~(1u << st)) | (par << st);
          next_stage();
        }
        w.next(p, n);
      }
      if (!ok) {
        if (!*s_abort) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x78000000u | (blockIdx.x & 0xFFFFFFu));
        *s_abort = 1u;
      }
      // every copy issued has landed before the CTA may leave
      for (int s = 0; s < C::kStages; ++s)
        if ((used >> s) & 1u) {
          uint32_t never = 0u;
          tc::mbar_wait(bar_full(s), (last >> s) & 1u, &never, 100000000ull);
        }
      for (int i = 0; i < 2; ++i)
        if ((qs >> i) & 1u) {                      // bar_q's parity follows bar_qfree's
          uint32_t never = 0u;
          tc::mbar_wait(bar_q(i), pqf[i], &never, 100000000ull);
        }
    } else if (warp == 8) {
      // ------------------------------------------------------------- MMAs
      const uint32_t q_desc = desc_k(s0 + C::kOffQ);
      auto mma_s = [&](int i, uint32_t kd) {
        const uint32_t qd = q_desc + i * (C::kTileB >> 4);
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb)
          mma_ss4(tm_s(i), qd + kb * (kTile * 128 >> 4), kd + kb * (kTile * 128 >> 4), C::kIdescS,
                  kb > 0);
        commit_elected(bar_s(i));
      };
      bool ok = true;
      uint32_t pq[2] = {0u, 0u}, pp[2] = {0u, 0u};   // parities of bar_q and bar_p
      while (ok && w.u < w.end) {
        int at;
        const int n = w.take(), nt = w.tiles(n, &at);
        const int nact = w.rp.n * g - w.mb * kRows > kTile ? 2 : 1;   // MMA tiles with rows
        if (nt > 0) {
          const int sk0 = st;
          ok = warp_wait(bar_full(sk0), par, s_abort);
          next_stage();
          const uint32_t kd0 = desc_k(s0 + sk0 * C::kTileB);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (i < nact && ok) {
              ok = warp_wait(bar_q(i), pq[i], s_abort);
              pq[i] ^= 1u;
              if (!ok) break;
              tc::tc_fence_after();
              mma_s(i, kd0);
            }
          if (ok) commit_elected(bar_empty(sk0));
        }
        for (int j = 0; ok && j < nt; ++j) {
          const bool more = j + 1 < nt;
          const int sv = st;
          ok = warp_wait(bar_full(sv), par, s_abort);
          next_stage();
          const int sk = st;
          if (more) {
            ok = ok && warp_wait(bar_full(sk), par, s_abort);
            next_stage();
          }
          const uint32_t vd = desc_mn(s0 + sv * C::kTileB), kd = desc_k(s0 + sk * C::kTileB);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i >= nact || !ok) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && warp_wait(bar_p(i, half), pp[i], s_abort);
              if (!ok) break;
              tc::tc_fence_after();
              mma_ts4(tm_o(i), tm_s(i) + half * 32, vd + half * (64 * 128 >> 4), C::kIdescO,
                      half > 0 ? 1u : (uint32_t)j);
            }
            if (!ok) break;
            pp[i] ^= 1u;
            if (more)
              mma_s(i, kd);
            else
              commit_elected(bar_s(i));   // O complete
          }
          if (!ok) break;
          commit_elected(bar_empty(sv));
          if (more) commit_elected(bar_empty(sk));
        }
        w.next(p, n);
      }
      if (!ok) {
        if (lane == 0 && !*s_abort)
          record_error(p.hdr, SDK_ERR_TIMEOUT, 0x79000000u | (blockIdx.x & 0xFFFFFFu));
        __syncwarp();
        *s_abort = 1u;
        // what was issued ends before TMEM is freed
        commit_elected(bar_done);
        uint32_t never = 0u;
        warp_wait(bar_done, 0u, &never, 100000000ull);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
    // --------------------------------------------------------------- softmax
    const int i = warp >> 2;
    const int rr = (warp & 3) * 32 + lane;         // row of the MMA tile, TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // out leaves by whole rows: D / 8 lanes of 16 bytes each
    constexpr int kLanesRow = D / 8, kRowsStep = 32 / kLanesRow, kSteps = 32 / kRowsStep;
    const int chunk = lane % kLanesRow, sub = lane / kLanesRow, wrow = (warp & 3) * 32;
    uint8_t* q_tile = smem + C::kOffQ + i * C::kTileB;   // out is staged there
    uint32_t ps = 0u;                              // parity of bar_s
    bool ok = true;
    Walk w = walk;
    if (tid == 0 && !p.whole) {
      Cut cut;
      cut.u0 = u0;
      cut.lo = cut_lo;
      cut.hi = cut_hi;
      cut.row0 = w.rp.row0;
      cut.rows = w.rp.n * g;
      cut.mb = w.mb;
      cut.h = w.h;
      reinterpret_cast<Cut*>(p.cuts)[blockIdx.x] = cut;
    }
#pragma unroll 1
    for (bool first = true; w.u < w.end; first = false) {
      int at;
      const int n = w.take(), nt = w.tiles(n, &at);
      const ReqPlan& rp = w.rp;
      const int rows = rp.n * g, r = w.mb * kRows + i * kTile + rr;   // packed row
      const int t_first = rp.lo + at * kTile;
      // partial sums: of the share's first segment or of its last
      const int slot = n < w.units() ? 2 * (int)blockIdx.x + (first ? 0 : 1) : -1;
      if (w.mb * kRows + i * kTile < rows && ok) {
        const bool live = r < rows;
        const int tok = live ? r / g : 0, hq = w.h * g + (live ? r - tok * g : 0);
        const int row = live ? (rp.row0 + tok) * p.Hq + hq : -1;
        // S c = log2 of the softmax term; rows past the last see nothing
        const float c = live ? __ldg(p.qscale + ((int64_t)(rp.pair0 + w.mb) * p.Hkv + w.h) * kRows +
                                     i * kTile + rr)
                             : 1.0f;
        const int pos = rp.len - rp.n + (live ? tok : (rows - 1) / g);
        const int see1 = p.causal ? min(pos, rp.len - 1) : rp.len - 1;     // last token seen
        const int see0 = p.window > 0 ? pos - p.window + 1 : 0;            // first one
        // tiles that lie within every row's sight need no mask
        const int w_hi = __reduce_min_sync(0xffffffffu, see1),
                  w_lo = __reduce_max_sync(0xffffffffu, see0);
        float m = -INFINITY, l = 0.0f;
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(bar_s(i), ps, s_abort));
          ps ^= 1u;
          if (!ok) break;
          tc::tc_fence_after();
          const int t0 = t_first + j * kTile;
          uint32_t v[4][32];
#pragma unroll
          for (int k = 0; k < 4; ++k) tc::tmem_ld32(tm_s(i) + lanes + k * 32, v[k]);
          tc::tmem_ld_wait();
          if (t0 + kTile - 1 > w_hi || t0 < w_lo) {
            const int lim1 = see1 - t0, lim0 = see0 - t0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int u = 0; u < 32; ++u)
                if (k * 32 + u > lim1 || k * 32 + u < lim0) v[k][u] = 0xFF800000u;   // -inf
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int u = 0; u < 32; u += 2)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = max3(mx[k], __uint_as_float(v[k][u]), __uint_as_float(v[k][u + 1]));
          const float mt = live ? fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c : -INFINITY;
          if (__any_sync(0xffffffffu, mt > m + kSlack)) {
            // lane by lane, so that a row's result does not hang on its neighbours'
            const float mn = mt > m + kSlack ? mt : m;
            const float f = m == mn ? 1.0f : ex2(m - mn);
            if (j > 0) {
              l *= f;
#pragma unroll
              for (int k = 0; k < D / 32; ++k) {
                uint32_t o[32];
                tc::tmem_ld32(tm_o(i) + lanes + k * 32, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                tmem_st32(tm_o(i) + lanes + k * 32, o);
              }
            }
            m = mn;
          }
          const float base = m == -INFINITY ? 0.0f : kPUp - m;
          const uint64_t c2 = pack2(c, c), base2 = pack2(base, base);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h2[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const uint64_t x = fma2(
                  pack2(__uint_as_float(v[k][2 * u]), __uint_as_float(v[k][2 * u + 1])), c2, base2);
              float y0, y1;
              if (u % kPolyOf == kPolyOf - 1) {
                ex2_fma(x, &y0, &y1);
              } else {
                unpack2(x, &y0, &y1);
                y0 = ex2(y0);
                y1 = ex2(y1);
              }
              sum[u & 1] = add2(sum[u & 1], pack2(y0, y1));
              const __half2 hh = __floats2half2_rn(y0, y1);
              h2[u] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            tmem_st16(tm_s(i) + lanes + k * 16, h2);
            if (k & 1) {   // 64 tokens of P are there: their product may begin
              tmem_st_wait();
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(bar_p(i, k >> 1));
            }
          }
          float l0, l1;
          unpack2(add2(sum[0], sum[1]), &l0, &l1);
          l += l0 + l1;
        }
        if (nt > 0 && ok) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(bar_s(i), ps, s_abort));
          ps ^= 1u;
          tc::tc_fence_after();
        }
        if (!ok && lane == 0) {
          if (!*s_abort)
            record_error(p.hdr, SDK_ERR_TIMEOUT, 0x7A000000u | (blockIdx.x & 0xFFFFFFu));
          *s_abort = 1u;
        }
        // m carries P's offset from here on: O and l are sums of 2^(x - m)
        const float mo = m == -INFINITY ? -INFINITY : m - kPUp;
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        if (live && ok) {
          if (slot >= 0)
            p.part_ml[(int64_t)slot * kRows + i * kTile + rr] = make_float2(mo, l);
          else if (p.lse != nullptr)
            p.lse[row] = l > 0.0f || l != l ? (mo + log2f(l)) * 0.69314718f : -INFINITY;
        }
        // whole rows go out through the free q tile; partial sums lie
        // [dim][row], as they come
        float* part = p.part_o + ((int64_t)slot * 2 + i) * D * kTile + rr;
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          if (nt > 0 && ok) {
            tc::tmem_ld32(tm_o(i) + lanes + k * 32, o);
            tc::tmem_ld_wait();
          } else {
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = 0u;
          }
          if (slot < 0 && nt > 0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 bb =
                    __floats2bfloat162_rn(__uint_as_float(o[8 * u + 2 * e]) * inv,
                                          __uint_as_float(o[8 * u + 2 * e + 1]) * inv);
                y[e] = *reinterpret_cast<const uint32_t*>(&bb);
              }
              *reinterpret_cast<uint4*>(q_tile + tile_off(rr, 4 * k + u)) =
                  make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (slot >= 0 && nt > 0 && live && ok) {
#pragma unroll
            for (int u = 0; u < 32; ++u) part[(k * 32 + u) * kTile] = __uint_as_float(o[u]);
          }
        }
        if (slot < 0 && ok) {
          __syncwarp();
#pragma unroll 4
          for (int k = 0; k < kSteps; ++k) {
            const int rk = __shfl_sync(0xffffffffu, row, k * kRowsStep + sub);
            if (rk >= 0)
              *(reinterpret_cast<uint4*>(p.out + (int64_t)rk * D) + chunk) =
                  nt > 0 ? *reinterpret_cast<const uint4*>(
                               q_tile + tile_off(wrow + k * kRowsStep + sub, chunk))
                         : make_uint4(0u, 0u, 0u, 0u);
          }
        }
        if (nt > 0) {                              // O is read, the q tile is free
          tc::fence_proxy_async();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar_qfree(i));
        }
      }
      w.next(p, n);
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

constexpr int kJoinRows = 32;      // rows of a block of chunk_join_kernel

// Joins the partial sums of the blocks of rows that several shares cut, in
// the shares' order.  Grid (share, part of the rows): share c stands for the
// block that its first unit lies inside of, if that is the first cut there.
// A lane takes a row, a warp D / 8 dims.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(ChunkParams p) {
  __shared__ float2 s_ml[kMaxShares * kJoinRows];
  pdl_wait();
  const Cut* cuts = reinterpret_cast<const Cut*>(p.cuts);
  const int c = (int)blockIdx.x + 1, shares = p.plan[p.B].npair;
  const Cut cut = cuts[c];                         // (of a share that is not there: not used)
  const int64_t before = cuts[c - 1].u0;
  if (c >= shares || cut.u0 == cut.lo || before > cut.lo) return;   // no cut, or an earlier one
  constexpr int E = D / 8;                         // dims a thread
  const int rb = blockIdx.y * kJoinRows + (threadIdx.x & 31), dim = threadIdx.x / 32 * E;
  const int r = cut.mb * kRows + rb;
  if (cut.mb * kRows + (int)blockIdx.y * kJoinRows >= cut.rows) return;
  // share c - 1 ends with its part, the shares c .. last start with theirs
  const int slot0 = 2 * (c - 1) + (before < cut.lo ? 1 : 0);
  auto slot = [&](int s) { return (int64_t)(s < c ? slot0 : 2 * s); };
  int last = c;
  while (last + 1 < shares && cuts[last + 1].u0 < cut.hi) ++last;
  const int parts = last - c + 2;                  // of the shares c - 1 .. last
  // the first two parts' sums are on their way while the weights are read
  auto sums_of = [&](int s) {
    return p.part_o + ((slot(c - 1 + s) * 2 + rb / kTile) * D + dim) * kTile + rb % kTile;
  };
  float x0[E], x1[E];
#pragma unroll
  for (int k = 0; k < E; ++k) {
    x0[k] = sums_of(0)[k * kTile];
    x1[k] = sums_of(1)[k * kTile];
  }
  for (int i = threadIdx.x; i < parts * kJoinRows; i += 256) {
    const int s = i / kJoinRows;
    s_ml[i] = p.part_ml[slot(c - 1 + s) * kRows + blockIdx.y * kJoinRows + i % kJoinRows];
  }
  __syncthreads();
  if (r >= cut.rows) return;
  const float2* ml = s_ml + (threadIdx.x & 31);
  float m = -INFINITY, z = 0.0f, o[E];
  for (int s = 0; s < parts; ++s) m = fmaxf(m, ml[s * kJoinRows].x);
  // what saw nothing left no sums: whatever is read there does not count
  auto weigh = [&](int s, bool* none) {
    const float2 w = ml[s * kJoinRows];
    *none = w.x == -INFINITY && w.y == 0.0f;
    const float f = *none ? 0.0f : ex2(w.x - m);
    z = fmaf(w.y, f, z);
    return f;
  };
  bool none0, none1;
  const float f0 = weigh(0, &none0), f1 = weigh(1, &none1);
#pragma unroll
  for (int k = 0; k < E; ++k) o[k] = fmaf(none1 ? 0.0f : x1[k], f1, none0 ? 0.0f : x0[k] * f0);
#pragma unroll 4
  for (int s = 2; s < parts; ++s) {
    const float* src = sums_of(s);
    bool none;
    const float f = weigh(s, &none);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float x = src[k * kTile];
      o[k] = fmaf(none ? 0.0f : x, f, o[k]);
    }
  }
  const int tok = r / p.g;
  const int64_t row = (int64_t)(cut.row0 + tok) * p.Hq + cut.h * p.g + (r - tok * p.g);
  const float inv = z > 0.0f || z != z ? 1.0f / z : 0.0f;
#pragma unroll
  for (int k = 0; k < E; k += 8) {
    uint32_t y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(o[k + 2 * e] * inv, o[k + 2 * e + 1] * inv);
      y[e] = *reinterpret_cast<const uint32_t*>(&a);
    }
    *reinterpret_cast<uint4*>(p.out + row * D + dim + k) = make_uint4(y[0], y[1], y[2], y[3]);
  }
  if (p.lse != nullptr && dim == 0)
    p.lse[row] = z > 0.0f || z != z ? (m + log2f(z)) * 0.69314718f : -INFINITY;
}

int64_t chunk_cap_tiles(int B, int max_len, int64_t total_len) {
  const int64_t each = (int64_t)B * ((max_len + (int64_t)kTile - 1) / kTile);
  if (total_len <= 0) return each;
  const int64_t sum = total_len / kTile + B;   // every context ends inside a tile at most once
  return sum < each ? sum : each;
}

// Which form a call takes, by what the three were measured to take (us; T:
// tokens times KV heads, half as much at head_dim 64).  Rebuilt for all:
// 34 and 0.84e-3 T, however many rows follow.  In one pass: 9.5 and 1e-3 T, a
// sixth more for 17 to 32 rows.  By atoms: a latency, the codes' way from HBM,
// the gathers and additions of every row pair, and the segments of every pair
// that an SM starts on.  32 query and 8 KV heads, us by tiles / in one pass /
// by atoms: one token over 256: 15 / 12 / 77; over 2048: 36 / 26 / 47; over
// 8192: 93 / 70 / 57; over 32768: 251 / 247 / 93; eight tokens over 2048: 36 /
// 32 / 91, over 32768: 245 / 289 / 238.
enum class Form { tiles, direct, atoms };
static Form pick_form(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q, int max_len,
                      int64_t total_len) {
  const int64_t q = max_q < n_tok ? max_q : n_tok, g = Hq / Hkv;
  if (q < 1) return Form::tiles;
  const double pairs = (double)((q * g + 1) / 2);
  const double all = min((double)B * pairs, (double)(n_tok * g + B) / 2) * Hkv;
  double T = (double)B * max_len;
  if (total_len > 0 && total_len < T) T = (double)total_len;
  T *= Hkv;
  const double dt = d == 128 ? T : 0.55 * T, tiles = 34 + 0.84e-3 * dt;
  const double direct = 9.5 + (q * g > 16 ? 1.17e-3 : 1e-3) * dt;
  const double atoms = 30 + 7e-5 * T + 4e-5 * T * pairs + 9.0 * n / SDK_MAX_ATOMS +
                       (15 + 22.0 * n / SDK_MAX_ATOMS) * all / num_sms();
  const bool one_pass = direct_fits(B, n_tok, (int)g, max_q, max_len) && direct < tiles;
  // by atoms, the pairs and the shares have to fit a grid, a pair's segments its join
  if (max_len <= kAtomsMaxLen && all <= (double)kAtomsMaxPairs && T * pairs <= (double)kAtomsMaxWork &&
      atoms < (one_pass ? direct : tiles) && tc::encode_fn() != nullptr)
    return Form::atoms;
  return one_pass ? Form::direct : Form::tiles;
}

// CTAs of the attention kernel.  Where the blocks fit the SMs, one for every
// part of a block, the parts of equal length (twelve mixed requests: 27.6 us, in
// equal shares 30.6 us: a share that ends one block and begins another fills
// and drains its pipeline twice), but whole blocks where no context is longer
// than 8 tiles and an eighth of the SMs have one (a prompt of 512 tokens, 64
// blocks: 26 us, in parts 31 us; 256 tokens over 444, 4 blocks: 24 us, in parts
// 20 us), or than 3 tiles (20 tokens of 200: 17.4 us, in parts 18.8 us; of 700:
// 26 and 24 us).  A CTA per block too where the blocks fill whole rounds of the SMs
// (their CTAs read a tile together; 2048 tokens over 32768, 256 blocks: 1250
// us, with shares 1300 us), else one per SM with equal shares.
struct ChunkCut {
  int ctas;
  bool whole, parts;
};
static ChunkCut chunk_cut(int64_t blocks, int Hkv, int max_len) {
  const int64_t tiles = (max_len + (int64_t)kTile - 1) / kTile, items = blocks * Hkv, sms = num_sms();
  const int64_t rounds = (items + sms - 1) / sms;
  int64_t most = min(sms, (int64_t)kMaxShares);
  ChunkCut c;
  c.parts = items <= most && blocks <= kRebThreads && (tiles > 8 || (tiles > 3 && 8 * items <= sms));
  c.whole = !c.parts && (rounds <= 1 ? tiles <= 8 : 5 * items >= 4 * rounds * sms);
  if (items > 0x7FFFFFFF) c.whole = false;
  if (c.whole) most = items;
  else if (c.parts) most = min(most, items * tiles);
  else if (items * (tiles + kBlockCost) < 4 * most) most = (items * (tiles + kBlockCost) + 3) / 4;
  c.ctas = (int)(most < 1 ? 1 : most);
  return c;
}

size_t chunk_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q,
                             int max_len, int64_t total_len) {
  const Form form = pick_form(B, n_tok, Hq, Hkv, d, n, max_q, max_len, total_len);
  if (form == Form::direct)
    return direct_workspace_bytes(B, n_tok, Hq, Hkv, d, max_q, max_len, total_len);
  if (form == Form::atoms)
    return atoms_workspace_bytes(B, n_tok, Hq, Hkv, d, n, max_q, max_len, total_len);
  const int64_t q = max_q < n_tok ? max_q : n_tok;
  const int64_t blocks = cap_blocks(B, n_tok, Hq / Hkv, (int)q);
  const ChunkCut c = chunk_cut(blocks, Hkv, max_len);
  return chunk_layout(B, blocks, Hkv, d, chunk_cap_tiles(B, max_len, total_len), c.ctas, c.whole)
      .total;
}

template <int D>
static sdk_status launch_d(const ChunkParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)2 * (p.B + 1) * 4;   // 33 KB at most: no opt-in
  static unsigned long long attr_set = 0ull;
  if (device_needs_setup(&attr_set)) {
    if (cudaFuncSetAttribute(chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ACfg<D>::kSmem) != cudaSuccess)
      return SDK_ERR_CUDA;
    device_setup_done(&attr_set);
  }
  // one kernel for everything, a step of tokens a warp, while neither the
  // tokens nor the rows are many (up to 4096 tokens and 40 rows of eight
  // requests: 38 against 41 us; a prompt of 4096 tokens: 63 against 54 us to
  // the end of the rebuilding)
  constexpr int kStep = 32 / (2 * (D / 8)) * (kRebThreads / 32);   // tokens of a CTA's step
  const int64_t steps = (int64_t)p.cap_tiles * p.Hkv * (kTile / kStep);
  constexpr int kPackRows = 32 / (D / 8) * kPackSteps * (kRebThreads / 32);   // rows of a CTA's step
  int64_t prep = (p.n_tok * p.Hq + kPackRows - 1) / kPackRows;
  if (prep > 4 * num_sms()) prep = 4 * num_sms();
  if (steps <= 80 * num_sms() && p.n_tok * p.Hq <= 32768) {
    // the plan's CTA and, since a tile has several steps, some more
    const int64_t grid = 1 + (steps < 2 * num_sms() - 1 ? steps : 2 * num_sms() - 1);
    rebuild_kernel<D, 1><<<(unsigned)grid, kRebThreads, smem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SDK_ERR_CUDA;
  } else {
    chunk_prep_kernel<D><<<(unsigned)prep, kRebThreads, smem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess ||
        launch_after(rebuild_kernel<D, 4>, dim3((unsigned)(8 * num_sms())), kRebThreads, smem, stream,
                     p) != cudaSuccess)
      return SDK_ERR_CUDA;
  }
  if (launch_after(chunk_attn_kernel<D>, dim3((unsigned)p.ctas), kAThreads, ACfg<D>::kSmem, stream,
                   p) != cudaSuccess)
    return SDK_ERR_CUDA;
  const int64_t most_rows = (int64_t)p.max_q * p.g < kRows ? (int64_t)p.max_q * p.g : kRows;
  if (p.ctas > 1 && !p.whole &&
      launch_after(chunk_join_kernel<D>,
                   dim3((unsigned)(p.ctas - 1), (unsigned)((most_rows + kJoinRows - 1) / kJoinRows)),
                   256, 0, stream, p) != cudaSuccess)
    return SDK_ERR_CUDA;
  return SDK_OK;
}

sdk_status launch_chunk_attn(ChunkParams p, int64_t total_len, char* workspace,
                             cudaStream_t stream) {
  p.hdr = reinterpret_cast<WsHeader*>(workspace);
  p.plan = reinterpret_cast<ReqPlan*>(workspace + sizeof(WsHeader));
  const Form form =
      pick_form(p.B, p.n_tok, p.Hq, p.Hkv, p.d, p.n, p.max_q, p.max_len, total_len);
  if (form == Form::direct) return launch_chunk_direct(p, total_len, workspace, stream);
  if (form == Form::atoms) return launch_chunk_atoms(p, total_len, workspace, stream);
  const int64_t blocks = cap_blocks(p.B, p.n_tok, p.g, p.max_q);
  p.cap_work = blocks;
  const ChunkCut c = chunk_cut(blocks, p.Hkv, p.max_len);
  p.ctas = c.ctas;
  p.whole = c.whole ? 1 : 0;
  p.parts = c.parts ? 1 : 0;
  const ChunkLayout l = chunk_layout(p.B, blocks, p.Hkv, p.d, p.cap_tiles, c.ctas, c.whole);
  p.cuts = workspace + l.cuts;
  p.units = reinterpret_cast<int64_t*>(workspace + l.units);
  p.qscale = reinterpret_cast<float*>(workspace + l.qs);
  p.qt = reinterpret_cast<__half*>(workspace + l.qt);
  p.kt = reinterpret_cast<__half*>(workspace + l.kt);
  p.vt = reinterpret_cast<__half*>(workspace + l.vt);
  p.part_ml = reinterpret_cast<float2*>(workspace + l.ml);
  p.part_o = reinterpret_cast<float*>(workspace + l.po);
  return p.d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace sdk
