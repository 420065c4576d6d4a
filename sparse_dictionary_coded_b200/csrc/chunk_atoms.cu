// Chunk attention (sdk_chunk_attn) for few rows over long contexts, by
// atoms instead of by rebuilt vectors:
//   <q, K_t> = sum_j c_tj <q, D_K[i_tj]>           scores by 16 gathers
//   sum_t p_t V_t = sum_a w_a D_V[a],  w_a = sum_t p_t sum_j c_tj [i_tj = a]
// so a row costs 16 gathers and 16 additions a token in shared memory
// (32768 atoms are 128 KB there), and the dictionaries are read once.
//   atoms_qd_kernel     QD = D_K q^T, tcgen05: atoms on M, rows on N; fp16,
//                       two rows side by side in one word per atom
//   atoms_token_kernel  scores, softmax and weights of its share of the
//                       (row pair, token) units, per segment of one pair
//   atoms_out_kernel    w D_V, tcgen05, atoms split over the CTAs
//   atoms_join_kernel   the segments' and atom ranges' sums, in fixed order
#include "chunk_plan.cuh"
#include "tc_ptx.cuh"

namespace sdk {

namespace {

constexpr int kN = 128;            // rows per MMA tile
constexpr int kM = 128;            // atoms per QD tile, head dims of w D_V
constexpr int kChunk = 64;         // atoms per step of w D_V
constexpr int kTab = SDK_MAX_ATOMS;
constexpr int64_t kShareTokens = 1 << 15;   // tokens of a share at most
// segments of a pair at most: shares are longer than half of kShareTokens
// where there are more of them than SMs
constexpr int kMaxSegs = 2 * (int)(kAtomsMaxLen / kShareTokens) + 2;
constexpr int kTokThreads = 640;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Shares that `work` units are cut into, none of them empty: of a thousand
// tokens at least (fewer would leave threads idle), one per SM, or as many for
// every SM as keep them within kShareTokens.  The host sizes the launch by the
// bound on the work, the device cuts the work there is: a share without a unit
// would leave its sums unwritten.
// A product p c is rounded to a unit of at most A / 5e8 (A = sum_t p_t sum_j
// |c_tj| over the share), so over S flat tokens its deviation is 9e-9 S of the
// mean product: 3e-4 at 2^15 tokens, below the 1e-3 that bf16 outputs have
// anyhow (without the bound 2e-3 at four requests of 262144).
__host__ __device__ __forceinline__ int share_count(int64_t work, int sms) {
  const int64_t want = work / 1024, rounds = (work + sms * kShareTokens - 1) / (sms * kShareTokens);
  return (int)(want < 1 ? 1 : want < sms ? want : sms * rounds);
}

struct AtomCut {
  int64_t pairs, work;             // bounds
  int ctas, row_tiles, ksplits, chunks, n_pad;
};

AtomCut atom_cut(int B, int64_t n_tok, int Hq, int Hkv, int n, int max_q, int max_len,
                 int64_t total_len) {
  AtomCut c;
  const int64_t g = Hq / Hkv, q = max_q < n_tok ? max_q : n_tok;
  const int64_t each = (q * g + 1) / 2;                    // pairs of one request and KV head
  c.pairs = (n_tok * g + B) / 2;                           // sum of ceil(n g / 2)
  if (c.pairs > each * B) c.pairs = each * B;
  c.pairs *= Hkv;
  int64_t tokens = (int64_t)B * max_len;
  if (total_len > 0 && total_len < tokens) tokens = total_len;
  c.work = tokens * Hkv * each;
  c.ctas = share_count(c.work, num_sms());
  // a segment is a CTA's share of one pair: at most ctas + pairs of them
  c.row_tiles = (int)((2 * (c.ctas + c.pairs) + kN - 1) / kN);
  c.chunks = (n + kChunk - 1) / kChunk;
  int ks = num_sms() / c.row_tiles;
  if (ks > c.chunks) ks = c.chunks;
  c.ksplits = ks < 1 ? 1 : ks;
  c.n_pad = (n + 3) / 4 * 4;                               // rows of QD in whole 16-byte pieces
  return c;
}

struct AtomLayout {
  size_t qd, scale, pair, score, ml, w, o, total;
};

AtomLayout atom_layout(int B, int d, const AtomCut& c) {
  AtomLayout l;
  const size_t rows = (size_t)c.row_tiles * kN;
  l.qd = up256(sizeof(WsHeader) + ((size_t)B + 1) * sizeof(ReqPlan));
  l.scale = up256(l.qd + (size_t)c.pairs * c.n_pad * 4);
  l.pair = up256(l.scale + (size_t)c.pairs * 8);
  l.score = up256(l.pair + (size_t)c.pairs * 16);
  l.ml = up256(l.score + (size_t)c.work * 8);
  l.w = up256(l.ml + rows * 8);
  l.o = up256(l.w + rows * c.chunks * kChunk * 2 * 2);
  l.total = up256(l.o + (size_t)c.ksplits * rows * d * 4);
  return l;
}

}  // namespace

// ------------------------------------------------------------------- QD

template <int D>
struct QdCfg {
  static constexpr int kStages = 3;
  static constexpr int kStageB = kM * D * 2;
  static constexpr int kOffB = kStages * kStageB;
  static constexpr int kOffBar = kOffB + kN * D * 2;
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffMax = kOffMisc + 16;         // [kN] largest |q| of a column's row
  static constexpr int kOffRow = kOffMax + kN * 4;      // [kN] its row of q, -1: none
  static constexpr int kOffUp = kOffRow + kN * 4;       // [kN] its scale
  static constexpr int kOffScan = kOffUp + kN * 4;      // [32] int64, then first pairs [B + 1]
  static constexpr int kSmem = kOffScan + 256 + (SDK_MAX_REQUESTS + 1) * 4 + 1024;
  static_assert(kSmem <= 232448, "exceeds the 227 KB shared memory of one sm_100 CTA");
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                     ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
};

// One CTA per (tile of 128 rows, strided set of 128-atom tiles): warp 0
// streams the dictionary by TMA, warp 1 issues the MMAs (bf16 atoms and
// queries, both exact, fp32 sums), warps 2-5 store.  A row is scaled by a
// power of two that puts its largest entry in [1, 2), so fp16 holds
// <q, d> with 11 significand bits for atoms of norm 1e-4 to 2900 (the rebuilt
// keys of the other forms are rounded as much; in fp32 a pair of rows would not
// fit the shared memory, and every token's words would be read twice as often).
// Bound by the read of D_K and, with many rows, the stores of QD.
template <int D>
__global__ void __launch_bounds__(192, 1)
    atoms_qd_kernel(const __grid_constant__ CUtensorMap kmap, ChunkParams p) {
  using C = QdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::align_smem_1k(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  uint32_t* s_max = reinterpret_cast<uint32_t*>(smem + C::kOffMax);
  int32_t* s_row = reinterpret_cast<int32_t*>(smem + C::kOffRow);
  float* s_up = reinterpret_cast<float*>(smem + C::kOffUp);
  int64_t* s_warp = reinterpret_cast<int64_t*>(smem + C::kOffScan);
  int32_t* s_pair0 = reinterpret_cast<int32_t*>(smem + C::kOffScan + 256);
  volatile uint32_t* s_abort = misc;
  volatile uint32_t* s_tmem = misc + 1;
  const uint32_t s0 = tc::smem_u32(smem);
  auto bar = [&](int i) { return tc::smem_u32(&bars[i]); };
  auto bar_full = [&](int s) { return bar(s); };
  auto bar_empty = [&](int s) { return bar(C::kStages + s); };
  auto bar_tfull = [&](int b) { return bar(2 * C::kStages + b); };
  auto bar_tempty = [&](int b) { return bar(2 * C::kStages + 2 + b); };
  const uint32_t bar_done = bar(2 * C::kStages + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_tiles = (p.n + kM - 1) / kM;
  pdl_launch();
  if (tid == 0) {
    *s_abort = 0u;
    for (int i = 0; i < C::kNumBars; ++i)
      tc::mbar_init(bar(i), i == 2 * C::kStages + 2 || i == 2 * C::kStages + 3 ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < kN) s_max[tid] = 0u;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tc::smem_u32((const void*)s_tmem)),
                 "r"(2 * kN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the first dictionary tiles are on their way while the plan is made
  auto load_tile = [&](int k) {
    const int st = k % C::kStages, a = blockIdx.x + k * gridDim.x;
    tc::mbar_expect_tx(bar_full(st), (uint32_t)C::kStageB);
#pragma unroll
    for (int kb = 0; kb < D / 64; ++kb)
      tc::tma_load_2d(s0 + st * C::kStageB + kb * (kM * 128), &kmap, kb * 64, a * kM, bar_full(st));
  };
  const int my_tiles = (n_tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  const int early = min(my_tiles, C::kStages);
  if (tid == 0)
    for (int k = 0; k < early; ++k) load_tile(k);
  make_plan<true>(p, blockIdx.x == 0 && blockIdx.y == 0, s_pair0, nullptr, s_warp);
  const int n_pairs = s_pair0[p.B];
  const int pair_base = blockIdx.y * (kN / 2);

  // the tile's query rows as the K-major B operand (zero past the last)
  if (tid < kN) {
    const int pair = pair_base + tid / 2;
    int row = -1;
    if (pair < n_pairs) {
      const int b = find_first(s_pair0, p.B, pair);
      const int row0 = p.cu_q[b], n = p.cu_q[b + 1] - row0;
      const int npair = (int)(((int64_t)n * p.g + 1) / 2);
      const int rel = pair - s_pair0[b], h = rel / npair;
      const int r = (rel - h * npair) * 2 + (tid & 1);
      if (r < n * p.g) {
        const int i = r / p.g;
        row = (row0 + i) * p.Hq + h * p.g + (r - i * p.g);
      }
    }
    s_row[tid] = row;
  }
  __syncthreads();
  {
    constexpr int kBatch = 4;    // loads in flight
    for (int e0 = tid; e0 < kN * (D / 8); e0 += kBatch * 192) {
      uint4 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int e = e0 + u * 192, row = e < kN * (D / 8) ? s_row[e / (D / 8)] : -1;
        v[u] = row < 0 ? make_uint4(0u, 0u, 0u, 0u)
                       : __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)row * D) + e % (D / 8));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int e = e0 + u * 192;
        if (e >= kN * (D / 8)) break;
        const int col = e / (D / 8), kc = e % (D / 8);
        uint32_t mx = 0u;
        const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = max(mx, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
        if (mx) atomicMax(&s_max[col], mx);
        *reinterpret_cast<uint4*>(smem + C::kOffB + (kc >> 3) * (kN * 128) + col * 128 +
                                  (((kc & 7) ^ (col & 7)) << 4)) = v[u];
      }
    }
  }
  tc::fence_proxy_async();
  __syncthreads();
  if (tid < kN) {
    // one factor does: where it is short of the row's scale (entries below
    // 2^-126) the scores vanish anyway
    float up, rest;
    row_scale(s_max[tid], 0, &up, &rest);
    s_up[tid] = up;
    const int other = __shfl_down_sync(0xffffffffu, s_row[tid], 1);
    if (blockIdx.x == 0 && pair_base + tid / 2 < n_pairs) {
      p.row_scale[2 * pair_base + tid] = p.scale * 1.44269504f / up;
      // the pair's rows; no shares so far
      if ((tid & 1) == 0) p.pair_of[pair_base + tid / 2] = make_int4(s_row[tid], other, 0, -1);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  if (pair_base < n_pairs) {   // else nothing but the totals
    if (warp == 0) {
      if (lane == 0) {
        bool ok = true;
        int k = early;
        for (; k < my_tiles; ++k) {
          const int st = k % C::kStages;
          if (!tc::mbar_wait(bar_empty(st), ((uint32_t)(k / C::kStages) & 1u) ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          load_tile(k);
        }
        if (!ok) {
          if (!*s_abort) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x60000000u | blockIdx.x);
          *s_abort = 1u;
        }
        for (int i = max(0, k - C::kStages); i < k; ++i) {   // copies in flight land first
          uint32_t never = 0u;
          tc::mbar_wait(bar_full(i % C::kStages), (uint32_t)(i / C::kStages) & 1u, &never,
                        100000000ull);
        }
      }
    } else if (warp == 1) {
      if (lane == 0) {
        bool ok = true;
        int k = 0;
        for (int a = blockIdx.x; a < n_tiles; a += gridDim.x, ++k) {
          const int st = k % C::kStages, tb = k & 1;
          if (!tc::mbar_wait(bar_full(st), (uint32_t)(k / C::kStages) & 1u, s_abort) ||
              !tc::mbar_wait(bar_tempty(tb), ((uint32_t)(k >> 1) & 1u) ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = (ks >> 2) * (kM * 128) + (ks & 3) * 32;
            tc::tc_mma(tmem + tb * kN, tc::smem_desc(s0 + st * C::kStageB + o),
                       tc::smem_desc(s0 + C::kOffB + o), C::kIdesc, ks > 0);
          }
          tc::tc_commit(bar_empty(st));
          tc::tc_commit(bar_tfull(tb));
        }
        if (!ok) {
          if (!*s_abort) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x61000000u | blockIdx.x);
          *s_abort = 1u;
        }
        tc::tc_commit(bar_done);
        uint32_t never = 0u;
        tc::mbar_wait(bar_done, 0u, &never, 100000000ull);
      }
      __syncwarp();
    } else {
      int k = 0;
      const int live = min(kN, 2 * (n_pairs - pair_base));
      for (int a = blockIdx.x; a < n_tiles; a += gridDim.x, ++k) {
        const int tb = k & 1;
        if (!__all_sync(0xffffffffu, tc::mbar_wait(bar_tfull(tb), (uint32_t)(k >> 1) & 1u, s_abort))) {
          if (lane == 0) {
            if (!*s_abort) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x62000000u | blockIdx.x);
            *s_abort = 1u;
          }
          break;
        }
        tc::tc_fence_after();
        const int quarter = warp & 3;
        const int atom = a * kM + quarter * 32 + lane;
        bool over = false;
        for (int cb = 0; cb < live; cb += 32) {
          uint32_t v[32];
          tc::tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + tb * kN + cb, v);
          tc::tmem_ld_wait();
          if (atom < p.n_pad) {
            __half2* dst = p.qd + (int64_t)(pair_base + cb / 2) * p.n_pad + atom;
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              if (cb + c >= live) break;
              const float2 up = *reinterpret_cast<const float2*>(s_up + cb + c);
              float x0 = __uint_as_float(v[c]) * up.x, x1 = __uint_as_float(v[c + 1]) * up.y;
              if (fmaxf(fabsf(x0), fabsf(x1)) > 65504.0f) {
                // infinities come from the query and stay
                over |= (fabsf(x0) > 65504.0f && !isinf(x0)) || (fabsf(x1) > 65504.0f && !isinf(x1));
                if (!isinf(x0)) x0 = fminf(fmaxf(x0, -65504.0f), x0 != x0 ? x0 : 65504.0f);
                if (!isinf(x1)) x1 = fminf(fmaxf(x1, -65504.0f), x1 != x1 ? x1 : 65504.0f);
              }
              dst[(int64_t)(c / 2) * p.n_pad] = __floats2half2_rn(x0, x1);
            }
          }
        }
        if (over) record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x64000000u | (uint32_t)atom);
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar_tempty(tb));
      }
    }
  }
  if (pair_base >= n_pairs && tid == 0)   // no rows here: the early copies land all the same
    for (int k = 0; k < early; ++k) {
      uint32_t never = 0u;
      tc::mbar_wait(bar_full(k), 0u, &never, 100000000ull);
    }
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kN)
                 : "memory");
  }
}

// ---------------------------------------------------------------- tokens

namespace {

constexpr uint32_t kNoRecord = 0xFFFFFFFFu;

// A token's position in the pages, stepped by kTokThreads without division.
struct PageAt {
  int col, off;
  __device__ void init(int t, int P) {
    col = t / P;
    off = t - col * P;
  }
  __device__ void step(int dcol, int doff, int P) {
    col += dcol;
    off += doff;
    if (off >= P) {
      off -= P;
      ++col;
    }
  }
};

// The page at `at`, -1 where not wanted; looked up two steps before its
// records are read.
__device__ __forceinline__ int page_of(const int32_t* table, const PageAt& at, bool wanted) {
  return wanted ? table[at.col] : -1;
}

// Index of the 128-byte record at offset `off` of a page for KV head h (all
// of them fit in 32 bits: 2^32 records are 512 GB), kNoRecord where not
// wanted or on a page outside the pool.
__device__ __forceinline__ uint32_t record_of(const ChunkParams& p, int page, int off, int h,
                                              bool wanted, int b) {
  if (!wanted) return kNoRecord;
  if (page < 0 || page >= p.n_pages) {
    record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x76000000u | (uint32_t)b);
    return kNoRecord;
  }
  return ((uint32_t)page * (uint32_t)p.Hkv + (uint32_t)h) * (uint32_t)p.page_size + (uint32_t)off;
}

// The lane's four words of the record that lane (l & ~3) | k holds; v: the
// value half.
__device__ __forceinline__ uint4 load_words(const ChunkParams& p, uint32_t rec, int k, int v) {
  const int lane = threadIdx.x & 31;
  const uint32_t r = __shfl_sync(0xffffffffu, rec, (lane & ~3) | k);
  if (r == kNoRecord) return make_uint4(0u, 0u, 0u, 0u);
  return __ldg(reinterpret_cast<const uint4*>(p.pages) + (int64_t)r * 8 + v * 4 + (lane & 3));
}

// Adds 2^x to the sum *z of terms over 2^*m, *m the largest x so far, with one
// exponential; kNone: none yet (below every score, but -inf).
constexpr float kNone = -3.4e38f;
__device__ __forceinline__ void add_term(float x, float* m, float* z) {
  const float d = x - *m, e = ex2(-fabsf(d));
  *z = d > 0.0f ? fmaf(*z, e, 1.0f) : *z + e;
  *m = fmaxf(*m, x);
}

template <typename F>
__device__ __forceinline__ float block_reduce(float v, float zero, float* s_red, F f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < kTokThreads / 32 ? s_red[threadIdx.x & 31] : zero;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A code word made harmless: NaN coefficients 0, infinite ones +-65504.
__device__ __forceinline__ uint32_t clean_word(uint32_t w, bool* bad) {
  if ((w & 0x7C000000u) != 0x7C000000u) return w;
  *bad = true;
  if (w & 0x03FF0000u) return w & 0x7FFFu;
  return (w & 0x80007FFFu) | 0x7BFF0000u;
}

// Adds p c of the segment's tokens [ta, ta + cnt) to the table for row e of
// the pair, with m the row's maximum and `up` the fixed point.  Returns this
// thread's part of sum_t p_t sum_j |c_tj|.  CLEAN: bad words are made harmless
// and recorded.  Tokens of no weight are not read.
template <bool FULL, bool CLEAN>
__device__ __forceinline__ float add_weights_of(const ChunkParams& p, uint32_t* tab,
                                                const float2* score, const int32_t* table, int h,
                                                int ta, int cnt, int e, float m, float up, int len,
                                                int b) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int own = (lane >> 2) + 8 * (lane & 3), mine = warp * 32 + own;
  const int P = p.page_size, dcol = kTokThreads / P, doff = kTokThreads - dcol * P;
  float sum = 0.0f;
  uint32_t top = 0u;
  auto score_of = [&](int u) {
    if (u >= cnt) return -INFINITY;
    const float2 s = score[u];
    return e ? s.y : s.x;
  };
  // words one step ahead, scores and pages two
  PageAt at;
  at.init(min(ta + mine, len), P);
  uint4 x[4], y[4];
  float w0 = ex2(score_of(mine) - m), s1 = score_of(mine + kTokThreads);
  const int pg0 = page_of(table, at, mine < cnt);
  const uint32_t rec0 = record_of(p, pg0, at.off, h, w0 > 0.0f, b);
  at.step(dcol, doff, P);
  int pg1 = page_of(table, at, mine + kTokThreads < cnt), off1 = at.off;
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = load_words(p, rec0, k, 1);
#pragma unroll 1
  for (int u = warp * 32; u < cnt; u += kTokThreads) {
    const float w1 = ex2(s1 - m);
    const uint32_t rec1 = record_of(p, pg1, off1, h, w1 > 0.0f, b);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = load_words(p, rec1, k, 1);
    at.step(dcol, doff, P);
    s1 = score_of(u + own + 2 * kTokThreads);
    pg1 = page_of(table, at, u + own + 2 * kTokThreads < cnt);
    off1 = at.off;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float pk = __shfl_sync(0xffffffffu, w0, (lane & ~3) | k);
      const float pu = pk * up;
      uint32_t ws[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      float ca = 0.0f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (CLEAN) ws[i] = clean_word(ws[i], &bad);
        const uint32_t a = word_idx(ws[i]);
        const float c = word_coef(ws[i]);
        ca += fabsf(c);
        atomicAdd(reinterpret_cast<int*>(tab) + a, __float2int_rn(pu * c));
        if (!FULL) top = max(top, a);
      }
      sum = fmaf(pk, ca, sum);
      if (CLEAN && bad) record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x77000000u | (uint32_t)b);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = y[k];
    w0 = w1;
  }
  if (!FULL && top >= (uint32_t)p.n)
    record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x77000000u | (uint32_t)b);
  return sum;
}

template <bool FULL>
__device__ __forceinline__ float add_weights(const ChunkParams& p, uint32_t* tab,
                                             const float2* score, const int32_t* table, int h,
                                             int ta, int cnt, int e, float m, float up, int len,
                                             int b) {
  return add_weights_of<FULL, false>(p, tab, score, table, h, ta, cnt, e, m, up, len, b);
}
// the rare way, kept out of the loop's registers
template <bool FULL>
__device__ __forceinline__ float add_clean_weights(const ChunkParams& p, uint32_t* tab,
                                                   const float2* score, const int32_t* table, int h,
                                                   int ta, int cnt, int e, float m, float up,
                                                   int len, int b) {
  return add_weights_of<FULL, true>(p, tab, score, table, h, ta, cnt, e, m, up, len, b);
}

}  // namespace

// A CTA, one at a time on an SM, takes an equal share of the (row pair, token)
// units, cut into segments of one pair.  Per segment:
//   1. QD of the pair (fp16, 128 KB) is copied to shared memory; a thread
//      per token adds up 16 gathered products for both rows at once and
//      keeps the scores in the workspace; the segment's maxima follow.
//   2. For each row the table becomes the weights: 16 integer additions a
//      token, p c in fixed point.  Integer sums make the result independent
//      of the order of the atomics.  The point puts A = sum_t p_t sum_j |c_tj|,
//      which bounds every atom's sum, near 10^9: A is estimated beforehand, as
//      the exact sum_t p_t times the mean |c| of 640 tokens spread over the
//      segment, weighted as they are; its exact value is summed up on the way,
//      and the row is redone with that where the estimate was off by more
//      than two: sums past 2^31 would wrap, small ones would lose bits.
//   3. The weights are written as two bf16 parts in the layout the product
//      with D_V reads: 16 significand bits, finer than the fixed point.
// One token for four requests of 32768: 127 us.  No unit is at its limit: the
// shared memory pipe is two thirds busy (random gathers and additions of 32
// lanes need 3.5 passes over the banks on average), the DRAM at 55 % of its
// peak (529 MB for 134 MB of codes: a pair reads the key words, each row of it
// the value words, and the pairs of a head at different times), and a share
// that ends one pair and begins another loads, clears and writes twice.
template <bool FULL>
__global__ void __launch_bounds__(kTokThreads, 1)
    atoms_token_kernel(const __grid_constant__ ChunkParams p) {
  extern __shared__ __align__(16) uint32_t tab[];   // [kTab]
  __shared__ float s_red[32];
  __shared__ float s_sample[kTokThreads / 32][6];
  __shared__ float s_bound[2], s_z[2];
  __shared__ __align__(8) uint64_t s_bar;
  __shared__ uint32_t s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int own = (lane >> 2) + 8 * (lane & 3), mine = warp * 32 + own;
  const int P = p.page_size;
  const int dcol = kTokThreads / P, doff = kTokThreads - dcol * P;
  pdl_launch();
  pdl_wait();
  const int64_t W = p.plan[p.B].work0;
  const int shares = share_count(W, p.sms);
  if (W == 0 || (int)blockIdx.x >= shares) return;
  int64_t w = W * blockIdx.x / shares;
  const int64_t w_end = W * (blockIdx.x + 1) / shares;
  int b;
  {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.plan[mid].work0 <= w) lo = mid; else hi = mid;
    }
    b = lo;
  }
  if (tid == 0) {
    s_abort = 0u;
    tc::mbar_init(tc::smem_u32(&s_bar), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  uint32_t parity = 0;
  auto fmax2 = [](float a, float c) { return fmaxf(a, c); };
  auto fadd2 = [](float a, float c) { return a + c; };
  while (w < w_end) {
    while (p.plan[b + 1].work0 <= w) ++b;     // p.plan[B] holds the totals
    const ReqPlan rp = p.plan[b];
    const int span = rp.len - rp.lo;
    const int64_t q = (w - rp.work0) / span;
    const int u0 = (int)(w - rp.work0 - q * span);
    const int cnt = (int)min((int64_t)(span - u0), w_end - w);
    const int h = (int)(q / rp.npair), j = (int)(q - (int64_t)h * rp.npair);
    const int pair = rp.pair0 + (int)q;
    const int slot = (int)blockIdx.x + pair;
    const int ta = rp.lo + u0, tb = ta + cnt;
    float2* score = p.score + w;
    if (tid == 0) {                           // the shares that hold the pair's tokens
      if (u0 == 0) p.pair_of[pair].z = (int)blockIdx.x;
      if (u0 + cnt == span) p.pair_of[pair].w = (int)blockIdx.x;
    }
    const int32_t* table = p.table + (int64_t)b * p.max_pages;

    tc::fence_proxy_async();
    __syncthreads();                          // the table is free
    if (tid == 0) {
      tc::mbar_expect_tx(tc::smem_u32(&s_bar), (uint32_t)p.n_pad * 4u);
      bulk_load(tc::smem_u32(tab), p.qd + (int64_t)pair * p.n_pad, (uint32_t)p.n_pad * 4u,
                tc::smem_u32(&s_bar));
    }
    if (!FULL)
      for (int a = p.n_pad + tid; a < kTab; a += kTokThreads) tab[a] = 0u;
    // what the two rows see
    int see0[2], see1[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * j + e, pos = rp.len - rp.n + r / p.g;
      const bool live = r < rp.n * p.g;
      see1[e] = !live ? -1 : p.causal ? min(pos, rp.len - 1) : rp.len - 1;
      see0[e] = p.window > 0 ? pos - p.window + 1 : 0;
    }
    const float sc0 = p.row_scale[2 * pair], sc1 = p.row_scale[2 * pair + 1];
    // sum_j |c_j| of the thread's sample of the values, on its way while QD is
    const int sampled = min(cnt, kTokThreads), sample = (int)((int64_t)tid * cnt / sampled);
    float sample_c = 0.0f;
    PageAt at;
    if (tid < sampled) {
      at.init(ta + sample, P);
      const uint32_t rec = record_of(p, page_of(table, at, true), at.off, h, true, b);
      if (rec != kNoRecord) {
        const uint4* words = reinterpret_cast<const uint4*>(p.pages) + (int64_t)rec * 8 + 4;
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = __ldg(words + k);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sample_c += (fabsf(word_coef(x[k].x)) + fabsf(word_coef(x[k].y))) +
                      (fabsf(word_coef(x[k].z)) + fabsf(word_coef(x[k].w)));
      }
    }
    const bool got = tc::mbar_wait(tc::smem_u32(&s_bar), parity, &s_abort);
    parity ^= 1u;
    if (!__syncthreads_and(got)) {
      if (tid == 0) {
        record_error(p.hdr, SDK_ERR_TIMEOUT, 0x65000000u | blockIdx.x);
        uint32_t never = 0u;                  // the copy lands before the CTA leaves
        tc::mbar_wait(tc::smem_u32(&s_bar), parity ^ 1u, &never, 100000000ull);
      }
      return;
    }

    // ---- scores.  A warp takes 32 tokens at a time; four lanes read one
    // token's record (64 contiguous bytes), lane l ends with the sums of
    // token own(l) = l / 4 + 8 (l % 4).
    float m0 = kNone, m1 = kNone, z0 = 0.0f, z1 = 0.0f;   // running maxima and sums of the lane's tokens
    bool nan0 = false, nan1 = false;
    uint32_t top = 0u;                        // largest atom index met
    // words one step ahead, pages two
    at.init(min(ta + mine, rp.len), P);
    uint4 x[4], y[4];
    uint32_t rec = record_of(p, page_of(table, at, mine < cnt), at.off, h, mine < cnt, b);
    at.step(dcol, doff, P);
    int pg1 = page_of(table, at, mine + kTokThreads < cnt), off1 = at.off;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = load_words(p, rec, k, 0);
#pragma unroll 1
    for (int u = warp * 32; u < cnt; u += kTokThreads) {
      const int t = ta + u + own;
      const uint32_t rec1 = record_of(p, pg1, off1, h, t + kTokThreads < tb, b);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = load_words(p, rec1, k, 0);
      at.step(dcol, doff, P);
      pg1 = page_of(table, at, t + 2 * kTokThreads < tb);
      off1 = at.off;
      float a[4][2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t ws[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        a[k][0] = a[k][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at_ = word_idx(ws[i]);
          const float2 qd = __half22float2(*reinterpret_cast<const __half2*>(tab + at_));
          const float c = word_coef(ws[i]);
          a[k][0] = fmaf(c, qd.x, a[k][0]);
          a[k][1] = fmaf(c, qd.y, a[k][1]);
          if (!FULL) top = max(top, at_);
        }
      }
      // sum over the four lanes, each keeping one token: first tokens k and
      // k ^ 1 change lanes, then k and k ^ 2
      float a0, a1;
      {
        const bool odd = lane & 1, high = lane & 2;
        float s[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const float give = odd ? a[2 * kk][e] : a[2 * kk + 1][e];
            const float keep = odd ? a[2 * kk + 1][e] : a[2 * kk][e];
            s[kk][e] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
          }
        a0 = (high ? s[1][0] : s[0][0]) +
             __shfl_xor_sync(0xffffffffu, high ? s[0][0] : s[1][0], 2);
        a1 = (high ? s[1][1] : s[0][1]) +
             __shfl_xor_sync(0xffffffffu, high ? s[0][1] : s[1][1], 2);
      }
      if (t < tb) {
        if (rec != kNoRecord && (!(fabsf(a0) < INFINITY) || !(fabsf(a1) < INFINITY))) {
          // a bad word, or a bad query row: the words are made harmless
          const uint32_t* words = p.pages + (int64_t)rec * 2 * kAtoms;
          bool bad = false;
          float b0 = 0.0f, b1 = 0.0f;
          for (int k = 0; k < kAtoms; ++k) {
            const uint32_t y = clean_word(__ldg(words + k), &bad);
            const float2 qd = __half22float2(*reinterpret_cast<const __half2*>(tab + word_idx(y)));
            b0 = fmaf(word_coef(y), qd.x, b0);
            b1 = fmaf(word_coef(y), qd.y, b1);
          }
          if (!(fabsf(a0) < INFINITY)) a0 = b0;
          if (!(fabsf(a1) < INFINITY)) a1 = b1;
          if (bad) record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x77000000u | (uint32_t)b);
        }
        a0 = t >= see0[0] && t <= see1[0] ? a0 * sc0 : -INFINITY;
        a1 = t >= see0[1] && t <= see1[1] ? a1 * sc1 : -INFINITY;
        nan0 |= a0 != a0;
        nan1 |= a1 != a1;
        add_term(a0, &m0, &z0);
        add_term(a1, &m1, &z1);
        score[t - ta] = make_float2(a0, a1);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = y[k];
      rec = rec1;
    }
    if (!FULL && top >= (uint32_t)p.n)
      record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x77000000u | (uint32_t)b);
    const bool row_nan0 = __syncthreads_or(nan0) != 0, row_nan1 = __syncthreads_or(nan1) != 0;
    const float q0 = block_reduce(m0, kNone, s_red, fmax2),
                q1 = block_reduce(m1, kNone, s_red, fmax2);
    z0 *= ex2(m0 - q0);
    z1 *= ex2(m1 - q1);
    m0 = q0 == kNone ? -INFINITY : q0;   // nothing seen
    m1 = q1 == kNone ? -INFINITY : q1;

    // ---- sum_t p_t, and the size of p c from one token per thread
    {
      float v[6] = {z0, 0.f, 0.f, z1, 0.f, 0.f};   // per row: sum of p; p and p |c| of the sample
      if (tid < sampled) {
        const float2 s2 = score[sample];
        const float p0 = ex2(s2.x - q0), p1 = ex2(s2.y - q1);
        if (p0 > 0.0f) v[1] = p0, v[2] = p0 * sample_c;            // (not for NaN)
        if (p1 > 0.0f) v[4] = p1, v[5] = p1 * sample_c;
      }
#pragma unroll
      for (int k = 0; k < 6; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < 6; ++k) s_sample[warp][k] = v[k];
      __syncthreads();
      if (tid < 2) {
        float t[3] = {0.f, 0.f, 0.f};
        for (int k = 0; k < kTokThreads / 32; ++k)
          for (int i = 0; i < 3; ++i) t[i] += s_sample[k][3 * tid + i];
        s_z[tid] = t[0];
        s_bound[tid] = t[1] > 0.0f ? t[0] * (t[2] / t[1]) : 0.0f;
      }
      __syncthreads();
    }

    // ---- weights, row by row
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      if (2 * j + e >= rp.n * p.g) break;
      const float m = e ? m1 : m0;
      const int row = 2 * slot + e;
      const bool isnan_row = e ? row_nan1 : row_nan0;
      if (isnan_row || m == -INFINITY || m == INFINITY) {
        // nothing seen (0), or a row that is NaN whatever its values are
        if (tid == 0)
          p.part_ml[row] = isnan_row || m == INFINITY
                               ? make_float2(0.0f, __int_as_float(0x7FC00000))
                               : make_float2(-INFINITY, 0.0f);
        continue;
      }
      float bound = s_bound[e], inv = 0.0f;
      bool clean = false;
#pragma unroll 1
      for (int attempt = 0; attempt < 3; ++attempt) {
        // (an estimate from bad words may be anything)
        const float up = 1.0e9f / fminf(fmaxf(bound, 1e-28f), 1e30f);
        inv = 1.0f / up;
        __syncthreads();
        for (int a = tid; a < kTab / 4; a += kTokThreads)
          reinterpret_cast<uint4*>(tab)[a] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        const float mine_aa =
            clean ? add_clean_weights<FULL>(p, tab, score, table, h, ta, cnt, e, m, up, rp.len, b)
                  : add_weights<FULL>(p, tab, score, table, h, ta, cnt, e, m, up, rp.len, b);
        const float aa = block_reduce(mine_aa, 0.0f, s_red, fadd2);
        if (aa * up < 2.0e9f && (aa * up > 5.0e8f || aa == 0.0f)) break;   // (false for NaN)
        if (aa < INFINITY)
          bound = aa;
        else
          clean = true;                       // a bad word; the third attempt knows A
      }
      __syncthreads();
      if (tid == 0) p.part_ml[row] = make_float2(m, s_z[e]);
      // [row tile][chunk][part][128 rows][64 atoms], 128-byte swizzle
      const int chunks = (p.n + kChunk - 1) / kChunk;
      char* img = p.wimg + (int64_t)(row / kN) * chunks * 2 * (kN * 128) + (row % kN) * 128;
      for (int o = tid; o < chunks * 8; o += kTokThreads) {
        const int4 v0 = reinterpret_cast<const int4*>(tab)[2 * o];
        const int4 v1 = reinterpret_cast<const int4*>(tab)[2 * o + 1];
        const int v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float f[2];
#pragma unroll
          for (int s = 0; s < 2; ++s)
            f[s] = FULL || 8 * o + 2 * u + s < p.n ? (float)v[2 * u + s] * inv : 0.0f;
          const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]);
          const __nv_bfloat162 c =
              __floats2bfloat162_rn(f[0] - __low2float(a), f[1] - __high2float(a));
          hi[u] = *reinterpret_cast<const uint32_t*>(&a);
          lo[u] = *reinterpret_cast<const uint32_t*>(&c);
        }
        char* dst = img + (int64_t)(o >> 3) * 2 * (kN * 128) + (((o & 7) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + kN * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    w += cnt;
  }
}

// ------------------------------------------------------------------ w D_V

struct OutCfg {
  static constexpr int kStages = 4;
  static constexpr int kA = kM * kChunk * 2;               // D_V chunk, two halves of 64 dims
  static constexpr int kB = 2 * kN * kChunk * 2;           // both parts of w
  static constexpr int kStage = kA + kB;
  static constexpr int kOffBar = kStages * kStage;
  static constexpr int kSmem = kOffBar + (2 * kStages + 1) * 8 + 16 + 1024;
  static_assert(kSmem <= 232448, "exceeds the 227 KB shared memory of one sm_100 CTA");
  // A (D_V) MN-major, B (w) K-major, both bf16
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) |
                                     ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
};

// out^T = D_V^T w^T for a tile of 128 rows over the CTA's atom range: head
// dims on M, rows on N, both operands by bulk and TMA copies; the partial
// sums go to the workspace.  Bound by the copies of w (4 bytes an atom and
// row) and D_V from L2.
template <int D>
__global__ void __launch_bounds__(128, 1)
    atoms_out_kernel(const __grid_constant__ CUtensorMap vmap, ChunkParams p) {
  using C = OutCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::align_smem_1k(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 2 * C::kStages + 1);
  volatile uint32_t* s_abort = misc;
  volatile uint32_t* s_tmem = misc + 1;
  const uint32_t s0 = tc::smem_u32(smem);
  auto bar_full = [&](int s) { return tc::smem_u32(&bars[s]); };
  auto bar_empty = [&](int s) { return tc::smem_u32(&bars[C::kStages + s]); };
  const uint32_t bar_done = tc::smem_u32(&bars[2 * C::kStages]);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch();
  pdl_wait();
  // rows that no segment wrote are not read
  const int rows = 2 * (share_count(p.plan[p.B].work0, p.sms) + p.plan[p.B].pair0);
  if ((int)blockIdx.y * kN >= rows) return;
  const int chunks = (p.n + kChunk - 1) / kChunk;
  const int c0 = (int)((int64_t)chunks * blockIdx.x / gridDim.x);
  const int c1 = (int)((int64_t)chunks * (blockIdx.x + 1) / gridDim.x);
  if (tid == 0) {
    *s_abort = 0u;
    for (int i = 0; i <= 2 * C::kStages; ++i) tc::mbar_init(tc::smem_u32(&bars[i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tc::smem_u32((const void*)s_tmem)),
                 "r"(kN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (D < kM) {
    // 64-dim heads: the upper half of every D_V stage stays zero
    for (int s = 0; s < C::kStages; ++s)
      for (int e = tid; e < C::kA / 32; e += 128)
        reinterpret_cast<uint4*>(smem + s * C::kStage + C::kA / 2)[e] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_proxy_async();
  }
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  if (warp == 0) {
    if (lane == 0) {
      const char* img = p.wimg + ((int64_t)blockIdx.y * chunks + c0) * C::kB;
      bool ok = true;
      int k = 0;
      for (; k < c1 - c0; ++k) {
        const int st = k % C::kStages;
        if (!tc::mbar_wait(bar_empty(st), ((uint32_t)(k / C::kStages) & 1u) ^ 1u, s_abort)) {
          ok = false;
          break;
        }
        const uint32_t sa = s0 + st * C::kStage;
        tc::mbar_expect_tx(bar_full(st), (uint32_t)(D * kChunk * 2 + C::kB));
        tc::tma_load_2d(sa, &vmap, 0, (c0 + k) * kChunk, bar_full(st));
        if (D > 64) tc::tma_load_2d(sa + C::kA / 2, &vmap, 64, (c0 + k) * kChunk, bar_full(st));
        bulk_load(sa + C::kA, img + (int64_t)k * C::kB, (uint32_t)C::kB, bar_full(st));
      }
      if (!ok) {
        if (!*s_abort) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x66000000u | blockIdx.x);
        *s_abort = 1u;
      }
      for (int i = max(0, k - C::kStages); i < k; ++i) {
        uint32_t never = 0u;
        tc::mbar_wait(bar_full(i % C::kStages), (uint32_t)(i / C::kStages) & 1u, &never,
                      100000000ull);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      for (int k = 0; k < c1 - c0; ++k) {
        const int st = k % C::kStages;
        if (!tc::mbar_wait(bar_full(st), (uint32_t)(k / C::kStages) & 1u, s_abort)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t sa = s0 + st * C::kStage, sb = sa + C::kA;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < kChunk / 16; ++ks)
            tc::tc_mma(tmem, tc::smem_desc_mn(sa + ks * 2048, C::kA / 2, 1024u),
                       tc::smem_desc(sb + part * (kN * 128) + ks * 32), C::kIdesc,
                       k > 0 || part > 0 || ks > 0);
        tc::tc_commit(bar_empty(st));
      }
      if (!ok) {
        if (!*s_abort) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x67000000u | blockIdx.x);
        *s_abort = 1u;
      }
      tc::tc_commit(bar_done);
    }
  }
  __syncwarp();
  uint32_t never = 0u;
  const bool done = __all_sync(0xffffffffu, tc::mbar_wait(bar_done, 0u, &never));
  if (!done && lane == 0) record_error(p.hdr, SDK_ERR_TIMEOUT, 0x68000000u | blockIdx.x);
  tc::tc_fence_after();
  const int dim = warp * 32 + lane;
  float* dst = p.part_o + ((int64_t)blockIdx.x * p.row_tiles + blockIdx.y) * kN * D + dim;
  if (done && warp * 32 < D) {
    for (int cb = 0; cb < kN && (int)blockIdx.y * kN + cb < rows; cb += 32) {
      uint32_t v[32];
      tc::tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + cb, v);
      tc::tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 32; ++c) dst[(int64_t)(cb + c) * D] = __uint_as_float(v[c]);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kN)
                 : "memory");
  }
}

// The sums of a row's segments over all atom ranges: a block takes 32 dims
// of a row, a thread per dim and group of partial sums, the groups joined in
// order.  Latency-bound: three dependent loads, those of a thread's sums in
// flight together.
template <int D>
__global__ void __launch_bounds__(512) atoms_join_kernel(ChunkParams p) {
  constexpr int G = 16;
  __shared__ float s_o[512];
  __shared__ float2 s_ml[kMaxSegs];
  pdl_wait();
  const int pair = (int)blockIdx.x / (2 * (D / 32)), e = (int)blockIdx.x / (D / 32) & 1;
  const int4 of = p.pair_of[pair];                 // (of a pair that is not there: not used)
  if (pair >= p.plan[p.B].pair0) return;
  const int row = e ? of.y : of.x;
  if (row < 0) return;                             // the pair has one row
  const int dim = (blockIdx.x % (D / 32)) * 32 + (threadIdx.x & 31), grp = threadIdx.x >> 5;
  const int c0 = of.z, segs = of.w - of.z + 1;     // 0: nothing to see
  const int64_t rows = (int64_t)p.row_tiles * kN, first = 2 * (int64_t)(c0 + pair) + e;
  float m = -INFINITY, z = 0.0f, o = 0.0f;
  for (int c = threadIdx.x; c < segs; c += 512) s_ml[c] = p.part_ml[first + 2 * c];
  __syncthreads();
  for (int c = 0; c < segs; ++c) m = fmaxf(m, s_ml[c].x);
  for (int c = 0; c < segs; ++c)
    if (s_ml[c].y != 0.0f) z = fmaf(s_ml[c].y, ex2(s_ml[c].x - m), z);
  const float* src = p.part_o + first * D + dim;
  const int all = segs * p.ksplits;
#pragma unroll 8
  for (int i = grp; i < all; i += G) {
    const int c = i / p.ksplits, k = i - c * p.ksplits;
    const float2 ml = s_ml[c];
    const float v = src[(k * rows + 2 * c) * D];
    // what saw nothing has no sums: whatever is read there does not count
    o = fmaf(ml.y != 0.0f ? ex2(ml.x - m) : 0.0f, ml.y != 0.0f ? v : 0.0f, o);
  }
  s_o[threadIdx.x] = o;
  __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int k = 1; k < G; ++k) o += s_o[k * 32 + threadIdx.x];
  const bool any = z > 0.0f || z != z;
  p.out[(int64_t)row * D + dim] =
      __bfloat16_as_ushort(__float2bfloat16_rn(z != z ? z : any ? o / z : 0.0f));
  if (p.lse != nullptr && dim == 0) p.lse[row] = any ? (m + log2f(z)) * 0.69314718f : -INFINITY;
}

// ------------------------------------------------------------------- host

size_t atoms_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q,
                             int max_len, int64_t total_len) {
  return atom_layout(B, d, atom_cut(B, n_tok, Hq, Hkv, n, max_q, max_len, total_len)).total;
}

template <int D>
static sdk_status launch_atoms_d(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                 const ChunkParams& p, cudaStream_t stream) {
  static unsigned long long attr_set = 0ull;
  if (device_needs_setup(&attr_set)) {
    if (cudaFuncSetAttribute(atoms_qd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             QdCfg<D>::kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(atoms_token_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kTab * 4) != cudaSuccess ||
        cudaFuncSetAttribute(atoms_token_kernel<false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kTab * 4) != cudaSuccess ||
        cudaFuncSetAttribute(atoms_out_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             OutCfg::kSmem) != cudaSuccess)
      return SDK_ERR_CUDA;
    device_setup_done(&attr_set);
  }
  const int tiles = (p.n + kM - 1) / kM;
  const unsigned ty = (unsigned)((2 * p.cap_pairs + kN - 1) / kN);
  unsigned gx = (unsigned)num_sms() / ty;
  gx = gx < 1 ? 1 : gx > (unsigned)tiles ? (unsigned)tiles : gx;
  atoms_qd_kernel<D><<<dim3(gx, ty), 192, QdCfg<D>::kSmem, stream>>>(kmap, p);
  if (cudaGetLastError() != cudaSuccess) return SDK_ERR_CUDA;
  const auto token = p.n == kTab ? atoms_token_kernel<true> : atoms_token_kernel<false>;
  if (launch_after(token, dim3((unsigned)p.ctas), kTokThreads, kTab * 4, stream, p) != cudaSuccess ||
      launch_after(atoms_out_kernel<D>, dim3((unsigned)p.ksplits, (unsigned)p.row_tiles), 128,
                   OutCfg::kSmem, stream, vmap, p) != cudaSuccess ||
      launch_after(atoms_join_kernel<D>, dim3((unsigned)(p.cap_pairs * 2 * (D / 32))), 512, 0,
                   stream, p) != cudaSuccess)
    return SDK_ERR_CUDA;
  return SDK_OK;
}

sdk_status launch_chunk_atoms(ChunkParams p, int64_t total_len, char* workspace,
                              cudaStream_t stream) {
  auto fn = tc::encode_fn();
  if (fn == nullptr) return SDK_ERR_CUDA;
  CUtensorMap maps[2];
  for (int s = 0; s < 2; ++s) {
    const cuuint64_t dims[2] = {(cuuint64_t)p.d, (cuuint64_t)p.n};
    const cuuint64_t strides[1] = {(cuuint64_t)p.d * 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)(s == 0 ? kM : kChunk)};
    const cuuint32_t estr[2] = {1u, 1u};
    if (fn(&maps[s], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
           const_cast<uint16_t*>(s == 0 ? p.dk : p.dv), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return SDK_ERR_CUDA;
  }
  const AtomCut c = atom_cut(p.B, p.n_tok, p.Hq, p.Hkv, p.n, p.max_q, p.max_len, total_len);
  const AtomLayout l = atom_layout(p.B, p.d, c);
  p.cap_pairs = c.pairs;
  p.cap_work = c.work;
  p.ctas = c.ctas;
  p.sms = num_sms();
  p.row_tiles = c.row_tiles;
  p.ksplits = c.ksplits;
  p.n_pad = c.n_pad;
  p.qd = reinterpret_cast<__half2*>(workspace + l.qd);
  p.row_scale = reinterpret_cast<float*>(workspace + l.scale);
  p.pair_of = reinterpret_cast<int4*>(workspace + l.pair);
  p.score = reinterpret_cast<float2*>(workspace + l.score);
  p.part_ml = reinterpret_cast<float2*>(workspace + l.ml);
  p.wimg = workspace + l.w;
  p.part_o = reinterpret_cast<float*>(workspace + l.o);
  return p.d == 128 ? launch_atoms_d<128>(maps[0], maps[1], p, stream)
                    : launch_atoms_d<64>(maps[0], maps[1], p, stream);
}

}  // namespace sdk
