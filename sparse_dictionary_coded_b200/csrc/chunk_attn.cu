// Attention of new tokens over paged codes (sdk_chunk_attn, include/sdk.h).
//
// Two kernels: rebuild_kernel writes the context's vectors
//   K_t = sum_j c_tj D_K[i_tj],  V_t = sum_j c_tj D_V[i_tj]
// once per call as fp16 tiles of 128 tokens in the workspace, and
// chunk_attn_kernel computes softmax(scale q K^T) V over the tiles.
#include "chunk_plan.cuh"
#include "tc_ptx.cuh"

namespace sdk {

namespace {

constexpr int kRebThreads = 256;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct ChunkLayout {
  size_t plan, kt, vt, ml, po, total;
};

ChunkLayout chunk_layout(int B, int64_t rows, int Hkv, int d, int64_t cap_tiles, int splits) {
  ChunkLayout l;
  const size_t tiles = (size_t)cap_tiles * Hkv * kTile * d * 2;
  l.plan = sizeof(WsHeader);
  l.kt = up256(l.plan + ((size_t)B + 1) * sizeof(ReqPlan));
  l.vt = l.kt + tiles;
  l.ml = l.vt + tiles;
  const size_t parts = splits > 1 ? (size_t)splits * rows : 0;
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

// The plan of the call and the rebuilt tiles.  Every CTA makes the plan
// itself (a scan over the requests' tile counts); CTA 0 leaves it in the
// workspace for the attention kernel.  D / 8 lanes rebuild one vector
// (16-byte pieces of an atom's row), a warp a token's key and value (two
// tokens at head_dim 64), TOK tokens one after the other with their code
// words read up front.  Bound by the gathers of 2 x 16 atom rows (8 KB per
// token and head at head_dim 128) from L2: 2.1 GB at 10.7 TB/s for 32768
// tokens of 8 heads.  With few tokens it is the chain of loads that counts,
// so there a warp takes one (TOK 1: 20.6 -> 11 us for eight short chats).
template <int D, int TOK>
__global__ void __launch_bounds__(kRebThreads) rebuild_kernel(ChunkParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_tile0 = sm;              // [B + 1]
  __shared__ int64_t s_warp[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch();
  make_plan<false>(p, blockIdx.x == 0, s_tile0, s_warp);

  constexpr int LPR = D / 8;           // lanes per record
  constexpr int TPS = 32 / (2 * LPR);  // tokens a warp rebuilds at a time
  constexpr int WPL = 16 / LPR;        // code words a lane holds
  constexpr int kItemTok = TOK * TPS * (kRebThreads / 32);   // tokens of a work item
  const int rec = lane / LPR, sub = lane % LPR;
  const int kv = rec & 1;
  const uint4* dict = reinterpret_cast<const uint4*>(kv ? p.dv : p.dk);
  char* tiles = reinterpret_cast<char*>(kv ? p.vt : p.kt);
  const int64_t items = (int64_t)s_tile0[p.B] * p.Hkv * (kTile / kItemTok);
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int part = (int)(it % (kTile / kItemTok));
    const int64_t th = it / (kTile / kItemTok);
    const int h = (int)(th % p.Hkv);
    const int tile = (int)(th / p.Hkv);
    const int b = find_first(s_tile0, p.B, tile);
    unsigned err;
    const ReqPlan rq = check_request(p, b, &err);
    const int t_tile = rq.lo + (tile - s_tile0[b]) * kTile;
    const int t_end = rq.n > 0 ? rq.len : 0;
    char* dst = tiles + ((int64_t)tile * p.Hkv + h) * (kTile * D * 2);
    const int r0 = part * kItemTok + warp * (TOK * TPS) + (rec >> 1);   // row of the tile
    uint32_t w[TOK][WPL];
    int page[TOK];
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      const int t = t_tile + r0 + u * TPS;
      page[u] = t < t_end ? p.table[(int64_t)b * p.max_pages + t / p.page_size] : -1;
    }
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      const int t = t_tile + r0 + u * TPS;
#pragma unroll
      for (int i = 0; i < WPL; ++i) w[u][i] = 0u;
      if (page[u] >= 0 && page[u] < p.n_pages) {
        const int off = t - t / p.page_size * p.page_size;
        const uint32_t* src =
            p.pages + ((((int64_t)page[u] * p.Hkv + h) * p.page_size + off) * 2 + kv) * kAtoms;
#pragma unroll
        for (int i = 0; i < WPL; ++i) w[u][i] = src[sub * WPL + i];
      } else if (t < t_end && sub == 0) {
        record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x76000000u | (uint32_t)b);
      }
    }
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      const int r = r0 + u * TPS;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      bool bad = false;
      if (t_tile + r - (rec >> 1) < t_end) {   // the warp's first token of the step
        uint4 v[kAtoms];
        float c[kAtoms];
#pragma unroll
        for (int j = 0; j < kAtoms; ++j) {
          const uint32_t x = __shfl_sync(0xffffffffu, w[u][j % WPL], rec * LPR + j / WPL);
          uint32_t a = word_idx(x);
          c[j] = word_coef(x);
          if (a >= (uint32_t)p.n) {
            bad = true;
            a = 0;
            c[j] = 0.0f;
          }
          v[j] = __ldg(dict + (int64_t)a * LPR + sub);
        }
#pragma unroll
        for (int j = 0; j < kAtoms; ++j) {
          acc[0] = fmaf(c[j], bf16_lo(v[j].x), acc[0]);
          acc[1] = fmaf(c[j], bf16_hi(v[j].x), acc[1]);
          acc[2] = fmaf(c[j], bf16_lo(v[j].y), acc[2]);
          acc[3] = fmaf(c[j], bf16_hi(v[j].y), acc[3]);
          acc[4] = fmaf(c[j], bf16_lo(v[j].z), acc[4]);
          acc[5] = fmaf(c[j], bf16_hi(v[j].z), acc[5]);
          acc[6] = fmaf(c[j], bf16_lo(v[j].w), acc[6]);
          acc[7] = fmaf(c[j], bf16_hi(v[j].w), acc[7]);
        }
      }
      // fp16 tiles: 11 significand bits (bf16 would have 8, and its
      // rounding of K, V and the probabilities would double the output's
      // error), the range the coefficients themselves have
      __half2 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x0 = acc[2 * i], x1 = acc[2 * i + 1];
        if (!(fabsf(x0) <= 65504.0f)) {
          bad = true;
          x0 = x0 != x0 ? 0.0f : copysignf(65504.0f, x0);
        }
        if (!(fabsf(x1) <= 65504.0f)) {
          bad = true;
          x1 = x1 != x1 ? 0.0f : copysignf(65504.0f, x1);
        }
        o[i] = __floats2half2_rn(x0, x1);
      }
      if (bad) record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x77000000u | (uint32_t)b);
      *reinterpret_cast<uint4*>(dst + tile_off(r, sub)) = *reinterpret_cast<const uint4*>(o);
    }
  }
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
// term: what 2^18 tokens lose by it is below 2^-13.
// q enters as fp16 scaled by a power of two per row (exact: 8 significand
// bits, the row's largest entry near 2^15).
// A context may be split over several CTAs (few rows, long contexts); their
// partial sums are joined by chunk_join_kernel.
namespace {

constexpr int kAThreads = 384;     // a warpgroup for each row tile, one of MMA and copy warps
// registers a thread after the split: 256 x 224 + 128 x 56 = 384 x 168, what
// the block is launched with (a row's 128 scores stay in registers)
constexpr int kRegsLaunch = 168, kRegsRows = 224, kRegsRest = 56;
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
  static constexpr int kNumBars = 2 * kStages + 2 + 4 + 2;
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
// own the issue was the bound (2048 tokens over 32768: 1084 us, so 916 us).
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
// Two floats in a register pair, for the two-wide fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
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
// (at most 2^-13.2, a fifth of the fp16 rounding that follows), n added to
// the exponent.  Below -127 the result is 0.
__device__ __forceinline__ void ex2_fma(uint64_t x2, float* y0, float* y1) {
  const float kBig = 12582912.0f;
  float a, b;
  unpack2(x2, &a, &b);
  x2 = pack2(fmaxf(a, -127.0f), fmaxf(b, -127.0f));
  const uint64_t t = add2(x2, pack2(kBig, kBig));
  const uint64_t n = add2(t, pack2(-kBig, -kBig));
  const uint64_t f = fma2(n, pack2(-1.0f, -1.0f), x2);
  uint64_t q = fma2(f, pack2(0.05500885908f, 0.05500885908f), pack2(0.2422110112f, 0.2422110112f));
  q = fma2(q, f, pack2(0.6932829447f, 0.6932829447f));
  q = fma2(q, f, pack2(1.0f, 1.0f));
  float t0, t1, q0, q1;
  unpack2(t, &t0, &t1);
  unpack2(q, &q0, &q1);
  *y0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
  *y1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
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

template <int D>
__global__ void __launch_bounds__(kAThreads, 1) chunk_attn_kernel(ChunkParams p) {
  using C = ACfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const int g = p.g;
  pdl_launch();
  pdl_wait();
  // the work item: consecutive CTAs share a KV head's tiles
  int w = blockIdx.x;
  const int split = w % p.splits;
  w /= p.splits;
  const int mb = p.mblocks - 1 - w % p.mblocks;   // the longest rows of a causal call first
  w /= p.mblocks;
  const int h = w % p.Hkv, b = w / p.Hkv;
  const ReqPlan rp = p.plan[b];
  const int rows = rp.n * g;                       // packed rows of this KV head
  const int r_base = mb * 2 * kTile;
  if (r_base >= rows) return;
  const int nact = rows - r_base > kTile ? 2 : 1;  // MMA tiles with rows

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
  const uint32_t bar_q = tc::smem_u32(&bars[2 * C::kStages + 6]);
  const uint32_t bar_done = tc::smem_u32(&bars[2 * C::kStages + 7]);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // tiles the block's rows see, and this split's share of them
  const int first_pos = rp.len - rp.n + r_base / g;
  const int last_row = min(r_base + 2 * kTile, rows) - 1;
  const int last_pos = rp.len - rp.n + last_row / g;
  const int t_hi = p.causal ? min(last_pos + 1, rp.len) : rp.len;
  const int t_lo = p.window > 0 ? max(0, first_pos - p.window + 1) : 0;
  int ta = 0, tb = 0;
  if (t_hi > t_lo) {
    const int a0 = (t_lo - rp.lo) / kTile, nt = (t_hi - rp.lo + kTile - 1) / kTile - a0;
    ta = a0 + (int)((int64_t)nt * split / p.splits);
    tb = a0 + (int)((int64_t)nt * (split + 1) / p.splits);
  }
  const int nt = tb - ta;

  if (tid == 0) {
    *s_abort = 0u;
    for (int s = 0; s < 2 * C::kStages + 2; ++s) tc::mbar_init(tc::smem_u32(&bars[s]), 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(bar_p(i >> 1, i & 1), 4);
    tc::mbar_init(bar_q, 4 * nact);
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

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 9 && lane == 0 && nt > 0) {
    // ------------------------------------------------------------- copies
      const char* kt = reinterpret_cast<const char*>(p.kt);
      const char* vt = reinterpret_cast<const char*>(p.vt);
      bool ok = true;
      int issued = 0;
      for (int k = 0; k < 2 * nt; ++k) {
        const int st = k % C::kStages;
        if (!tc::mbar_wait(bar_empty(st), ((uint32_t)(k / C::kStages) & 1u) ^ 1u, s_abort)) {
          ok = false;
          break;
        }
        const int64_t tile = (int64_t)(rp.tile0 + ta + (k >> 1)) * p.Hkv + h;
        tc::mbar_expect_tx(bar_full(st), (uint32_t)C::kTileB);
        bulk_load(s0 + st * C::kTileB, ((k & 1) ? vt : kt) + tile * C::kTileB, (uint32_t)C::kTileB,
                  bar_full(st));
        issued = k + 1;
      }
      if (!ok) {
        if (!*s_abort) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x78000000u | (blockIdx.x & 0xFFFFFFu));
        *s_abort = 1u;
      }
      // every copy issued has landed before the CTA may leave
      for (int k = max(0, issued - C::kStages); k < issued; ++k) {
        uint32_t never = 0u;
        tc::mbar_wait(bar_full(k % C::kStages), (uint32_t)(k / C::kStages) & 1u, &never, 100000000ull);
      }
    }
    if (warp == 8 && nt > 0) {
    // --------------------------------------------------------------- MMAs
      bool ok = warp_wait(bar_q, 0u, s_abort);
      // the ring's next stage and its parity
      int st = 0;
      uint32_t par = 0;
      auto next = [&]() {
        if (++st == C::kStages) {
          st = 0;
          par ^= 1u;
        }
      };
      const uint32_t q_desc = desc_k(s0 + C::kOffQ);
      auto mma_s = [&](int i, uint32_t kd) {
        const uint32_t qd = q_desc + i * (C::kTileB >> 4);
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb)
          mma_ss4(tm_s(i), qd + kb * (kTile * 128 >> 4), kd + kb * (kTile * 128 >> 4), C::kIdescS,
                  kb > 0);
        commit_elected(bar_s(i));
      };
      ok = ok && warp_wait(bar_full(0), 0u, s_abort);
      if (ok) {
        tc::tc_fence_after();
        const uint32_t kd = desc_k(s0);
        mma_s(0, kd);
        if (nact > 1) mma_s(1, kd);
        commit_elected(bar_empty(0));
      }
      next();
      for (int j = 0; ok && j < nt; ++j) {
        const bool more = j + 1 < nt;
        const int sv = st;
        ok = warp_wait(bar_full(sv), par, s_abort);
        next();
        const int sk = st;
        if (more) {
          ok = ok && warp_wait(bar_full(sk), par, s_abort);
          next();
        }
        const uint32_t vd = desc_mn(s0 + sv * C::kTileB), kd = desc_k(s0 + sk * C::kTileB);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i >= nact || !ok) break;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && warp_wait(bar_p(i, half), (uint32_t)j & 1u, s_abort);
            if (!ok) break;
            tc::tc_fence_after();
            mma_ts4(tm_o(i), tm_s(i) + half * 32, vd + half * (64 * 128 >> 4), C::kIdescO,
                    half > 0 ? 1u : (uint32_t)j);
          }
          if (!ok) break;
          if (more)
            mma_s(i, kd);
          else
            commit_elected(bar_s(i));   // O complete
        }
        if (!ok) break;
        commit_elected(bar_empty(sv));
        if (more) commit_elected(bar_empty(sk));
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
    if ((warp >> 2) < nact) {
    // ------------------------------------------------------------ softmax
    const int i = warp >> 2;
    const int rr = (warp & 3) * 32 + lane;         // row of the MMA tile, TMEM lane
    const int r = r_base + i * kTile + rr;         // packed row
    const bool live = r < rows;
    const int tok = live ? r / g : 0, hq = h * g + (live ? r - tok * g : 0);
    const int64_t row = (int64_t)(rp.row0 + tok) * p.Hq + hq;
    float c;                                       // S c = log2 of the softmax term
    {
      uint4 v[D / 8];
      const uint4* src = reinterpret_cast<const uint4*>(p.q + row * D);
#pragma unroll
      for (int k = 0; k < D / 8; ++k) v[k] = live ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
      uint32_t mx = 0u;                            // largest |q| as bf16 bits
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int u = 0; u < 4; ++u) mx = max(mx, max(x[u] & 0x7FFFu, (x[u] >> 16) & 0x7FFFu));
      }
      float up, up2;
      row_scale(mx, 14, &up, &up2);
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const __half2 hh = __floats2half2_rn(bf16_lo(x[u]) * up * up2, bf16_hi(x[u]) * up * up2);
          y[u] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        *reinterpret_cast<uint4*>(smem + C::kOffQ + i * C::kTileB + tile_off(rr, k)) =
            make_uint4(y[0], y[1], y[2], y[3]);
      }
      c = p.scale * 1.44269504f / up / up2;
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar_q);
    }
    const int pos = rp.len - rp.n + (live ? tok : last_row / g);
    const int see1 = p.causal ? min(pos, rp.len - 1) : rp.len - 1;     // last token seen
    const int see0 = p.window > 0 ? pos - p.window + 1 : 0;            // first one
    // tiles that lie within every row's sight need no mask
    const int w_hi = __reduce_min_sync(0xffffffffu, see1), w_lo = __reduce_max_sync(0xffffffffu, see0);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait(bar_s(i), (uint32_t)j & 1u, s_abort));
      if (!ok) break;
      tc::tc_fence_after();
      const int t0 = rp.lo + (ta + j) * kTile;
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
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
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
          const uint64_t x =
              fma2(pack2(__uint_as_float(v[k][2 * u]), __uint_as_float(v[k][2 * u + 1])), c2, base2);
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
      ok = __all_sync(0xffffffffu, tc::mbar_wait(bar_s(i), (uint32_t)nt & 1u, s_abort));
      tc::tc_fence_after();
    }
    if (!ok && lane == 0) {
      if (!*s_abort) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x7A000000u | (blockIdx.x & 0xFFFFFFu));
      *s_abort = 1u;
    }
    // m carries P's offset from here on: O and l are sums of 2^(x - m)
    const float mo = m == -INFINITY ? -INFINITY : m - kPUp;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    if (p.splits == 1 && p.lse != nullptr && live && ok)
      p.lse[row] = l > 0.0f || l != l ? (mo + log2f(l)) * 0.69314718f : -INFINITY;
    if (p.splits > 1 && live && ok) {
      p.part_ml[(int64_t)split * p.n_tok * p.Hq + row] = make_float2(mo, l);
    }
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
      if (live && ok) {
        if (p.splits == 1) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + row * D + k * 32);
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
            dst[u] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(
              p.part_o + ((int64_t)split * p.n_tok * p.Hq + row) * D + k * 32);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
      }
    }
    tc::tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// Joins the splits' partial sums, one warp per (row, query head).
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(ChunkParams p) {
  constexpr int E = D / 32;
  pdl_wait();
  const int64_t R = p.n_tok * p.Hq;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  // rows of no request, or of a refused one, stay as they were
  const int tok = (int)(row / p.Hq);
  const ReqPlan rp = p.plan[find_request(p, tok)];
  if (row >= R || tok < rp.row0 || tok >= rp.row0 + rp.n) return;
  float m = -INFINITY;
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, p.part_ml[s * R + row].x);
  float z = 0.0f, o[E];
#pragma unroll
  for (int k = 0; k < E; ++k) o[k] = 0.0f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = p.part_ml[s * R + row];
    if (ml.x == -INFINITY && ml.y == 0.0f) continue;   // saw nothing
    const float f = ex2(ml.x - m);
    z = fmaf(ml.y, f, z);
    const float* src = p.part_o + (s * R + row) * D + lane * E;
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = fmaf(src[k], f, o[k]);
  }
  const bool any = z > 0.0f || z != z;
#pragma unroll
  for (int k = 0; k < E; ++k)
    p.out[row * D + lane * E + k] = __bfloat16_as_ushort(__float2bfloat16_rn(any ? o[k] / z : 0.0f));
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = any ? (m + log2f(z)) * 0.69314718f : -INFINITY;
}

// How the call is cut: row blocks per request and KV head, and splits of
// the contexts.  A context is split while the blocks do not fill the SMs,
// down to four tiles a split (below that the copies' latency and the join
// outweigh what more CTAs bring).
struct ChunkCut {
  int mblocks, splits;
};
static ChunkCut chunk_cut(int B, int64_t n_tok, int Hq, int Hkv, int max_q, int max_len,
                          int window) {
  const int g = Hq / Hkv;
  const int64_t q = max_q < n_tok ? max_q : n_tok;
  ChunkCut c;
  c.mblocks = (int)((q * g + 2 * kTile - 1) / (2 * kTile));
  int64_t blocks = n_tok * g / (2 * kTile) + B;
  if (blocks > (int64_t)B * c.mblocks) blocks = (int64_t)B * c.mblocks;
  blocks *= Hkv;
  int64_t span = max_len;
  if (window > 0 && window + q < span) span = window + q;
  const int64_t tiles = (span + kTile - 1) / kTile;
  int64_t s = blocks > 0 ? num_sms() / blocks : 1;
  if (s > tiles / 4) s = tiles / 4;
  c.splits = (int)(s < 1 ? 1 : s);
  return c;
}

int64_t chunk_cap_tiles(int B, int max_len, int64_t total_len) {
  const int64_t each = (int64_t)B * ((max_len + (int64_t)kTile - 1) / kTile);
  if (total_len <= 0) return each;
  const int64_t sum = total_len / kTile + B;   // every context ends inside a tile at most once
  return sum < each ? sum : each;
}

// Which form a call takes.  Rebuilding costs 0.74 ns a token and KV head
// (head_dim 128), however many rows follow; going by atoms costs PER_PAIR
// for every two rows and FIXED once.
static bool by_atoms(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q, int max_len,
                     int64_t total_len) {
  const int64_t q = max_q < n_tok ? max_q : n_tok;
  const int64_t pairs = (q * (Hq / Hkv) + 1) / 2;
  const int64_t tokens = (total_len > 0 ? total_len : (int64_t)B * max_len) * Hkv;
  if (q < 1) return false;
  return pairs <= 8 && tokens >= 65536;
}

size_t chunk_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q,
                             int max_len, int64_t total_len) {
  // without a window: a window only lowers the number of splits
  const ChunkCut c = chunk_cut(B, n_tok, Hq, Hkv, max_q, max_len, 0);
  const size_t a =
      chunk_layout(B, n_tok * Hq, Hkv, d, chunk_cap_tiles(B, max_len, total_len), c.splits).total;
  if (!by_atoms(B, n_tok, Hq, Hkv, d, n, max_q, max_len, total_len)) return a;
  const size_t b = atoms_workspace_bytes(B, n_tok, Hq, Hkv, d, n, max_q, max_len, total_len);
  return a > b ? a : b;
}

template <int D>
static sdk_status launch_d(const ChunkParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)(p.B + 1) * 4;
  static unsigned long long attr_set = 0ull;
  if (device_needs_setup(&attr_set)) {
    if (cudaFuncSetAttribute(chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ACfg<D>::kSmem) != cudaSuccess)
      return SDK_ERR_CUDA;
    device_setup_done(&attr_set);
  }
  // a warp takes one step of tokens where that many warps are not more than
  // the device holds at once, else four
  constexpr int kStep = 32 / (2 * (D / 8)) * (kRebThreads / 32);   // tokens of a CTA's step
  const int64_t steps = (int64_t)p.cap_tiles * p.Hkv * (kTile / kStep);
  int64_t grid;
  if (steps <= 8 * num_sms()) {
    grid = steps;
    rebuild_kernel<D, 1><<<(unsigned)grid, kRebThreads, smem, stream>>>(p);
  } else {
    grid = steps / 4 < 8 * num_sms() ? steps / 4 : 8 * num_sms();
    rebuild_kernel<D, 4><<<(unsigned)grid, kRebThreads, smem, stream>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return SDK_ERR_CUDA;
  const int64_t ctas = (int64_t)p.B * p.Hkv * p.mblocks * p.splits;
  if (ctas > 0x7FFFFFFF) return SDK_ERR_INVALID_ARG;
  if (launch_after(chunk_attn_kernel<D>, dim3((unsigned)ctas), kAThreads, ACfg<D>::kSmem, stream,
                   p) != cudaSuccess)
    return SDK_ERR_CUDA;
  if (p.splits > 1 && launch_after(chunk_join_kernel<D>, dim3((unsigned)((p.n_tok * p.Hq + 7) / 8)),
                                   256, 0, stream, p) != cudaSuccess)
    return SDK_ERR_CUDA;
  return SDK_OK;
}

sdk_status launch_chunk_attn(ChunkParams p, int64_t total_len, char* workspace,
                             cudaStream_t stream) {
  p.hdr = reinterpret_cast<WsHeader*>(workspace);
  p.plan = reinterpret_cast<ReqPlan*>(workspace + sizeof(WsHeader));
  if (by_atoms(p.B, p.n_tok, p.Hq, p.Hkv, p.d, p.n, p.max_q, p.max_len, total_len)) {
    bool taken = false;
    const sdk_status s = launch_chunk_atoms(p, total_len, workspace, stream, &taken);
    if (taken) return s;
  }
  const ChunkCut c = chunk_cut(p.B, p.n_tok, p.Hq, p.Hkv, p.max_q, p.max_len, p.window);
  const ChunkLayout l = chunk_layout(p.B, p.n_tok * p.Hq, p.Hkv, p.d, p.cap_tiles, c.splits);
  p.mblocks = c.mblocks;
  p.splits = c.splits;
  p.kt = reinterpret_cast<__half*>(workspace + l.kt);
  p.vt = reinterpret_cast<__half*>(workspace + l.vt);
  p.part_ml = reinterpret_cast<float2*>(workspace + l.ml);
  p.part_o = reinterpret_cast<float*>(workspace + l.po);
  return p.d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace sdk
