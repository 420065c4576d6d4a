// The plan of a chunk attention call, made on the device from the requests'
// lengths: checked bounds and running sums, the same for every CTA.
#pragma once

#include "paged.cuh"

namespace sdk {

constexpr int kTile = 128;   // tokens of a rebuilt tile; the first one a request sees rounds down to one
constexpr int kRows = 256;   // packed rows of a block: two MMA tiles

// Inclusive scan of one 64-bit value per thread (blockDim.x a multiple of
// 32, <= 1024).
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t* s_warp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t t = lane < nw ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    if (lane < nw) s_warp[lane] = t;
  }
  __syncthreads();
  const int64_t r = warp > 0 ? v + s_warp[warp - 1] : v;
  *total = s_warp[nw - 1];
  __syncthreads();
  return r;
}

// The first token that a row of a request sees: its first row stands at len - n.
// Tokens before it are neither looked up in the table nor read (their pages may
// serve others by now).
__device__ __forceinline__ int first_seen(const ChunkParams& p, int len, int n) {
  return p.window > 0 ? (int)max((int64_t)len - n - p.window + 1, (int64_t)0) : 0;
}

// Checks request b's offsets and lengths; n = 0 refuses it (err says why).
__device__ __forceinline__ ReqPlan check_request(const ChunkParams& p, int b, unsigned* err) {
  ReqPlan r = {};
  r.row0 = p.cu_q[b];
  const int row1 = p.cu_q[b + 1];
  r.len = p.lens[b];
  *err = 0;
  if (r.row0 < 0 || row1 < r.row0 || row1 > p.n_tok || r.len < 0)
    *err = SDK_ERR_DEVICE_CHECK;
  else if (row1 - r.row0 > p.max_q || r.len > p.max_len)
    *err = SDK_ERR_CAPACITY;
  else
    r.n = row1 - r.row0;
  if (r.n > 0) {
    r.lo = min(first_seen(p, r.len, r.n), r.len) / kTile * kTile;
    r.ntiles = (r.len - r.lo + kTile - 1) / kTile;
    r.npair = (int)(((int64_t)r.n * p.g + 1) / 2);
  }
  return r;
}

// Scans all requests.  s_first [B + 1]: first tile (ATOMS: first row pair)
// of every request, s_block [B + 1] (not ATOMS): its first block of packed
// rows; the leader CTA leaves the plan and its totals in the workspace.  A
// request whose tiles or blocks (ATOMS: row pairs or work) pass what the host's
// bounds gave room for is refused (offsets that fall count rows twice).
template <bool ATOMS>
__device__ void make_plan(const ChunkParams& p, bool leader, int32_t* s_first, int32_t* s_block,
                          int64_t* s_warp) {
  const int64_t cap = ATOMS ? p.cap_pairs : p.cap_tiles;
  int64_t first = 0, work = 0;
  __shared__ unsigned long long s_used, s_work;   // what the accepted requests take
  if (threadIdx.x == 0) {
    s_first[0] = 0;
    if (!ATOMS) s_block[0] = 0;
    s_used = s_work = 0ull;
  }
  __syncthreads();
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    unsigned err = 0;
    ReqPlan r = {};
    if (b < p.B) r = check_request(p, b, &err);
    if (ATOMS && r.n > 0) r.lo = min(first_seen(p, r.len, r.n), r.len);
    const int64_t units = ATOMS ? (int64_t)r.npair * p.Hkv : r.ntiles;
    int64_t tot_u, tot_w = 0;
    const int64_t upto = first + block_scan64(units, s_warp, &tot_u);
    // units of work (ATOMS), or blocks of rows
    const int64_t mine = ATOMS ? units * (r.len - r.lo) : ((int64_t)r.n * p.g + kRows - 1) / kRows;
    const int64_t done = work + block_scan64(mine, s_warp, &tot_w);
    if (b < p.B) {
      // once over, the sums stay over: every later request with units is
      // refused too, and the totals end with the last accepted one
      if ((units > 0 || mine > 0) && (upto > cap || done > p.cap_work)) {
        err = SDK_ERR_CAPACITY;
        r.n = 0;
      } else if (leader && units > 0) {
        atomicMax(&s_used, (unsigned long long)upto);
        atomicMax(&s_work, (unsigned long long)done);
      }
      if (!ATOMS) s_block[b + 1] = (int)min(done, p.cap_work);
      s_first[b + 1] = (int)min(upto, cap);
      if (leader) {
        r.tile0 = (int)min(upto - units, cap);
        if (ATOMS) {
          r.pair0 = r.tile0;
          r.work0 = min(done - mine, p.cap_work);
        } else {
          r.pair0 = (int)min(done - mine, p.cap_work);
          r.npair = (int)mine;
        }
        if (r.n == 0) r.ntiles = r.npair = 0;
        p.plan[b] = r;
        if (err) record_error(p.hdr, err, 0x75000000u | (uint32_t)b);
      }
    }
    first += tot_u;
    work += tot_w;
  }
  __syncthreads();
  if (leader && threadIdx.x == 0) {
    // p.plan[B]: the totals
    ReqPlan t = {};
    t.pair0 = t.tile0 = (int)s_used;
    t.work0 = (int64_t)s_work;
    p.plan[p.B] = t;
  }
}

// The last b in [0, B) with first[b] <= e.
__device__ __forceinline__ int find_first(const int32_t* first, int B, int e) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= e) lo = mid; else hi = mid;
  }
  return lo;
}

// The request whose rows hold row `tok` of q (one of them; the caller checks).
__device__ __forceinline__ int find_request(const ChunkParams& p, int tok) {
  return find_first(p.cu_q, p.B, tok);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^e for a row of bf16 bits with largest magnitude mx (as bits) so that its
// largest entry's exponent becomes `to` (e = 0 for a row of zeros, or one
// with infinities or NaN, which spoil that row alone), as two factors that
// are each in float's range.
__device__ __forceinline__ void row_scale(uint32_t mx, int to, float* a, float* b) {
  int e = (mx >> 7) == 255u || mx == 0u ? 0 : to + 127 - (int)max(mx >> 7, 1u);
  *a = __uint_as_float((uint32_t)(min(e, 126) + 127) << 23);
  *b = __uint_as_float((uint32_t)(max(e - 126, 0) + 127) << 23);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
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

// Lane `sub` of the D / 8 that rebuild record `rec` of the warp: its eight
// entries of sum_j c_j dict[i_j] as fp16.  w: the lane's 16 / (D / 8) code
// words; ALL: all 16 atoms' rows in flight.  bad: an atom not in the
// dictionary (it counts as 0) or an entry out of range.
template <int D, bool ALL>
__device__ __forceinline__ uint4 rebuild_piece(const ChunkParams& p, const uint4* dict,
                                               const uint32_t (&w)[128 / D], int rec, int sub,
                                               bool* bad) {
  constexpr int LPR = D / 8, WPL = 16 / LPR;
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
  auto word = [&](int j) { return __shfl_sync(0xffffffffu, w[j % WPL], rec * LPR + j / WPL); };
  auto add = [&](float c, const uint4& v) {
    const uint64_t cc = pack2(c, c);
    acc[0] = fma2(cc, pack2(bf16_lo(v.x), bf16_hi(v.x)), acc[0]);
    acc[1] = fma2(cc, pack2(bf16_lo(v.y), bf16_hi(v.y)), acc[1]);
    acc[2] = fma2(cc, pack2(bf16_lo(v.z), bf16_hi(v.z)), acc[2]);
    acc[3] = fma2(cc, pack2(bf16_lo(v.w), bf16_hi(v.w)), acc[3]);
  };
  auto atom = [&](uint32_t x) {
    const uint32_t a = word_idx(x);
    if (a >= (uint32_t)p.n) *bad = true;
    return a < (uint32_t)p.n ? a : 0u;
  };
  auto coef = [&](uint32_t x) { return word_idx(x) < (uint32_t)p.n ? word_coef(x) : 0.0f; };
  if (ALL) {
    uint4 v[kAtoms];
#pragma unroll
    for (int j = 0; j < kAtoms; ++j) v[j] = __ldg(dict + (int64_t)atom(word(j)) * LPR + sub);
#pragma unroll
    for (int j = 0; j < kAtoms; ++j) add(coef(word(j)), v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kAtoms; ++j) {
      const uint32_t x = word(j);
      add(coef(x), __ldg(dict + (int64_t)atom(x) * LPR + sub));
    }
  }
  // fp16: 11 significand bits (bf16 would have 8, and its rounding of K, V
  // and the probabilities would double the output's error), the range the
  // coefficients themselves have
  __half2 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x0, x1;
    unpack2(acc[i], &x0, &x1);
    if (!(fabsf(x0) <= 65504.0f)) {
      *bad = true;
      x0 = x0 != x0 ? 0.0f : copysignf(65504.0f, x0);
    }
    if (!(fabsf(x1) <= 65504.0f)) {
      *bad = true;
      x1 = x1 != x1 ? 0.0f : copysignf(65504.0f, x1);
    }
    o[i] = __floats2half2_rn(x0, x1);
  }
  return *reinterpret_cast<const uint4*>(o);
}

// Launches a kernel that may start while its predecessor in the stream
// drains; the kernel itself waits (pdl_wait) before it touches global memory.
template <class... KArgs, class... Args>
inline cudaError_t launch_after(void (*kern)(KArgs...), dim3 grid, int block, size_t smem,
                                cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace sdk
