// Chunk attention (sdk_chunk_attn) for few rows over short contexts, in one
// pass: a CTA rebuilds 32 tokens' keys and values
//   K_t = sum_j c_tj D_K[i_tj],  V_t = sum_j c_tj D_V[i_tj]
// as fp16 in shared memory and attends to them at once, with a running
// maximum and sum per row, so that nothing but the partial sums of contexts
// that several CTAs share goes through the workspace.
//   chunk_direct_kernel       all contexts, in parts of equal length
//   chunk_direct_join_kernel  the sums of contexts in several parts
// What counts here is the chain of dependent loads: lengths, page, code words,
// atoms' rows (16 in flight a lane).
#include "chunk_plan.cuh"
#include "tc_ptx.cuh"

namespace sdk {

namespace {

constexpr int kDirThreads = 256, kDirWarps = kDirThreads / 32;
constexpr int kUnit = 16;          // tokens of a unit of work
constexpr int kStep = 32;          // tokens rebuilt and attended to at a time
constexpr int kMaxParts = 512;     // CTAs, and parts of a context
constexpr int kJoinRows = 8;       // blocks that share a context's rows when joining, at least
constexpr float kUp = 14.0f;       // log2 of P's offset: its smallest fp16 step is 2^-38 of the largest term

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// A context of one KV head in several parts, left for the join.
struct Split {
  int row0, rows, h, parts, slot;
};

struct DirectLayout {
  size_t splits, ml, po, total;
};

DirectLayout direct_layout(int rows, int d, int ctas) {
  DirectLayout l;
  l.splits = up256(sizeof(WsHeader) + sizeof(ReqPlan));
  // a context in parts of S units has at most 2 u / S, so all of them at
  // most twice as many parts as there are CTAs, and half as many contexts
  l.ml = up256(l.splits + (size_t)ctas * sizeof(Split));
  l.po = up256(l.ml + (size_t)2 * ctas * rows * 8);
  l.total = up256(l.po + (size_t)2 * ctas * rows * d * 4);
  return l;
}

int pad_rows(int64_t rows) { return rows <= 16 ? 16 : 32; }

// Two CTAs per SM, or one for every unit there can be.
int direct_ctas(int B, int Hkv, int max_len, int64_t total_len) {
  int64_t units = (int64_t)B * (max_len / kUnit + 2);
  if (total_len > 0 && total_len / kUnit + 2 * (int64_t)B < units) units = total_len / kUnit + 2 * (int64_t)B;
  units *= Hkv;
  const int most = 2 * num_sms() < kMaxParts ? 2 * num_sms() : kMaxParts;
  return (int)(units < most ? units : most);
}

// Four 8x8 matrices of halves from shared memory, rows at the lanes' addresses.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const __half* at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(tc::smem_u32(at)) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], const __half* at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(tc::smem_u32(at)) : "memory");
}
// c += a b: 16 rows, 8 columns, 16 deep
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace

// Every CTA looks over the requests itself (at most one per thread): the
// contexts are cut into parts of S units of 16 tokens, S the smallest length
// that leaves no more parts than CTAs (shares of exactly equal length made
// some CTAs walk the chain of loads twice: drafts of eight requests 24.6 us).
// The products are small (32 tokens and 16 or 32 rows at a time), so the
// warps' own matrix instructions do them; P and the sums as in chunk_attn.cu.
template <int D, int MT>
__global__ void __launch_bounds__(kDirThreads, 2) chunk_direct_kernel(ChunkParams p) {
  constexpr int kR = MT * 16;          // rows, padded
  constexpr int kPitch = D + 8;        // halves of a row: 16 bytes off the banks' period
  constexpr int LPR = D / 8;           // lanes per record
  constexpr int TPS = 32 / (2 * LPR);  // tokens a warp rebuilds at a time
  constexpr int WPL = 16 / LPR;        // code words a lane holds
  constexpr int NU = kStep / (TPS * kDirWarps);   // times a step
  constexpr int kNT = D / 8 / kDirWarps;          // O column tiles of a warp
  constexpr int kRW = kR / kDirWarps;             // rows whose softmax a warp does
  __shared__ __align__(16) __half s_q[kR * kPitch];
  __shared__ __align__(16) __half s_k[kStep * kPitch];
  __shared__ __align__(16) __half s_v[2][kStep * kPitch];
  __shared__ __align__(16) __half s_p[kR * (kStep + 8)];
  __shared__ float s_s[kR * (kStep + 1)];
  __shared__ float s_c[kR], s_f[kR], s_m[kR], s_l[kR];
  __shared__ int4 s_req[kDirThreads];             // row0, n, len, first token
  __shared__ int s_units[kDirThreads], s_tiles[kDirThreads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch();

  // ---- the plan, by every warp for itself
  if (tid < p.B) {
    unsigned err;
    const ReqPlan rq = check_request(p, tid, &err);
    int lo = 0, units = 0;
    if (rq.n > 0) {
      // the first token any row sees, rounded down to a unit
      lo = min(first_seen(p, rq.len, rq.n), rq.len) / kUnit * kUnit;
      units = max((rq.len - lo + kUnit - 1) / kUnit, 1);
    }
    s_req[tid] = make_int4(rq.row0, rq.n, rq.len, lo);
    s_units[tid] = units;
    s_tiles[tid] = rq.ntiles;
    if (err && blockIdx.x == 0) record_error(p.hdr, err, 0x75000000u | (uint32_t)tid);
  }
  __syncthreads();
  auto sum_of = [&](auto f) {          // of all requests
    int v = 0;
    for (int r = lane; r < p.B; r += 32) v += f(r);
    return __reduce_add_sync(0xffffffffu, v);
  };
  // tiles of 128 tokens are what the caller's bound on the lengths is held
  // against, as in the other form
  if (sum_of([&](int r) { return s_tiles[r]; }) > p.cap_tiles) {
    __syncthreads();
    if (tid == 0) {
      int64_t tiles = 0;
      for (int r = 0; r < p.B; ++r) {
        tiles += s_tiles[r];
        if (tiles > p.cap_tiles && s_units[r] > 0) {
          s_units[r] = 0;
          if (blockIdx.x == 0) record_error(p.hdr, SDK_ERR_CAPACITY, 0x75000000u | (uint32_t)r);
        }
      }
    }
    __syncthreads();
  }
  const int U = sum_of([&](int r) { return s_units[r]; });       // per KV head
  const int room = max((int)gridDim.x / p.Hkv, 1);               // parts per KV head
  int S = max((int)((uint32_t)(U + room - 1) / (uint32_t)room), 1), items;
  float per_s;
  // ceil(units / S); exact, the quotient is half a unit off whole numbers and
  // units are at most 2^16
  auto parts_of = [&](int r) { return (int)(((float)(s_units[r] + S) - 0.5f) * per_s); };
  for (int i = 0;; ++i) {
    per_s = __frcp_rn((float)S);
    items = sum_of(parts_of);
    if (items <= room || i == 8) break;            // (more requests than CTAs: several parts each)
    S += (S + 7) / 8;
  }

  if (blockIdx.x == 0 && warp == 0) {
    const int splits = sum_of([&](int r) { return parts_of(r) > 1 ? 1 : 0; });
    if (lane == 0) p.plan[0].npair = splits * p.Hkv;
  }
  const int rec = lane / LPR, sub = lane % LPR, kv = rec & 1;
  const uint4* dict = reinterpret_cast<const uint4*>(kv ? p.dv : p.dk);
  int buf = 0;
#pragma unroll 1
  for (uint32_t item = blockIdx.x; item < (uint32_t)(items * p.Hkv); item += gridDim.x) {
    // part `part` of request b's context, for KV head h
    const int h = (int)(item % (uint32_t)p.Hkv);
    int part = (int)(item / (uint32_t)p.Hkv), b = 0, parts = 0, before = 0, split = 0;   // split parts, contexts before b's
    for (int r0 = 0;; r0 += 32) {
      const int mine = r0 + lane < p.B ? parts_of(r0 + lane) : 0;
      int upto = mine;
#pragma unroll
      for (int e = 1; e < 32; e <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, e);
        if (lane >= e) upto += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, upto > part);
      const int at = past ? __ffs(past) - 1 : 32;
      before += __reduce_add_sync(0xffffffffu, lane < at && mine > 1 ? mine : 0);
      split += __popc(__ballot_sync(0xffffffffu, lane < at && mine > 1));
      if (past) {
        b = r0 + at;
        parts = __shfl_sync(0xffffffffu, mine, at);
        part -= __shfl_sync(0xffffffffu, upto, at) - parts;
        break;
      }
      part -= __shfl_sync(0xffffffffu, upto, 31);
    }
    const int4 r4 = s_req[b];
    const int row0 = r4.x, n = r4.y, len = r4.z, rows = n * p.g;
    const int t_begin = r4.w + part * S * kUnit, t_end = min(len, t_begin + S * kUnit);
    const int t_seen = first_seen(p, len, n);
    const int slot = parts > 1 ? before * p.Hkv + h * parts + part : -1;
    if (parts > 1 && part == 0 && tid == 0) {
      Split c;
      c.row0 = row0;
      c.rows = rows;
      c.h = h;
      c.parts = parts;
      c.slot = slot;
      reinterpret_cast<Split*>(p.cuts)[split * p.Hkv + h] = c;
    }
    // code words of the step at t0: the warp's tokens t0 + warp TPS, and so on
    uint32_t w[NU][WPL];
    auto load_words = [&](int t0) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int t = t0 + (i * kDirWarps + warp) * TPS + (rec >> 1);
#pragma unroll
        for (int k = 0; k < WPL; ++k) w[i][k] = 0u;
        if (t >= t_seen && t < t_end) {   // (tokens before the first seen one are zero)
          const int col = t / p.page_size, off = t - col * p.page_size;
          const int page = p.table[(int64_t)b * p.max_pages + col];
          if (page >= 0 && page < p.n_pages) {
            const uint32_t* src =
                p.pages + ((((int64_t)page * p.Hkv + h) * p.page_size + off) * 2 + kv) * kAtoms;
#pragma unroll
            for (int k = 0; k < WPL; ++k) w[i][k] = src[sub * WPL + k];
          } else if (sub == 0) {
            record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x76000000u | (uint32_t)b);
          }
        }
      }
    };
    load_words(t_begin);

    // the rows of q, fp16 scaled by a power of two that puts the row's
    // largest entry near 2^15 (exact: 8 significand bits)
#pragma unroll
    for (int r0 = 0; r0 < kR; r0 += kDirThreads / LPR) {
      const int r = r0 + tid / LPR, c8 = tid % LPR, tok = r / p.g;
      if (r0 + kDirThreads / LPR > kR && r >= kR) break;   // (whole warps)
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows)
        v = __ldg(reinterpret_cast<const uint4*>(
                      p.q + ((int64_t)(row0 + tok) * p.Hq + h * p.g + (r - tok * p.g)) * D) + c8);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      uint32_t mx = 0u, y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mx = max(mx, max(x[k] & 0x7FFFu, (x[k] >> 16) & 0x7FFFu));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float up, up2;
      row_scale(mx, 14, &up, &up2);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 hh = __floats2half2_rn(bf16_lo(x[k]) * up * up2, bf16_hi(x[k]) * up * up2);
        y[k] = *reinterpret_cast<const uint32_t*>(&hh);
      }
      *reinterpret_cast<uint4*>(s_q + r * kPitch + c8 * 8) = make_uint4(y[0], y[1], y[2], y[3]);
      if (c8 == 0) s_c[r] = p.scale * 1.44269504f / up / up2;
    }

    float m[kRW], l[kRW];              // of rows warp + 8 i; l: the lane's part
#pragma unroll
    for (int i = 0; i < kRW; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
    }
    float o[MT][kNT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < kNT; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][k][e] = 0.0f;

#pragma unroll 1
    for (int t0 = t_begin; ; t0 += kStep) {
      const bool last = t0 + kStep >= t_end;
      // ---- keys and values of 32 tokens; those behind the share's are zero
#pragma unroll 1
      for (int i = 0; i < NU; ++i) {               // (unrolled, the code itself is slow to come)
        const int r = (i * kDirWarps + warp) * TPS + (rec >> 1);
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (t0 + r - (rec >> 1) < t_end) {
          bool bad = false;
          y = rebuild_piece<D, true>(p, dict, w[0], rec, sub, &bad);
          if (bad) record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x77000000u | (uint32_t)b);
        }
        *reinterpret_cast<uint4*>((kv ? s_v[buf] : s_k) + r * kPitch + sub * 8) = y;
#pragma unroll
        for (int j = 1; j < NU; ++j)
#pragma unroll
          for (int k = 0; k < WPL; ++k) w[j - 1][k] = w[j][k];
      }
      if (!last) load_words(t0 + kStep);
      __syncthreads();
      // ---- scores: a 16 x 8 tile a warp and round
#pragma unroll
      for (int j0 = 0; j0 < MT * (kStep / 8); j0 += kDirWarps) {
        const int j = j0 + warp, mt = j / (kStep / 8), nt = j % (kStep / 8);
        if (MT * (kStep / 8) < kDirWarps && mt >= MT) break;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < D; k += 32) {
          uint32_t a0[4], a1[4], kk[4];
          ldsm4(a0, s_q + (mt * 16 + (lane & 15)) * kPitch + k + (lane >> 4) * 8);
          ldsm4(a1, s_q + (mt * 16 + (lane & 15)) * kPitch + k + 16 + (lane >> 4) * 8);
          ldsm4(kk, s_k + (nt * 8 + (lane & 7)) * kPitch + k + (lane >> 3) * 8);
          mma16(s, a0, kk[0], kk[1]);
          mma16(s, a1, kk[2], kk[3]);
        }
        float* dst = s_s + (mt * 16 + (lane >> 2)) * (kStep + 1) + nt * 8 + (lane & 3) * 2;
        dst[0] = s[0];
        dst[1] = s[1];
        dst[8 * (kStep + 1)] = s[2];
        dst[8 * (kStep + 1) + 1] = s[3];
      }
      __syncthreads();
      // ---- softmax: a lane is a token
#pragma unroll
      for (int i = 0; i < kRW; ++i) {
        const int r = warp + i * kDirWarps;
        float y = 0.0f, f = 1.0f;
        if (r < rows) {
          const int t = t0 + lane, pos = len - n + r / p.g;
          const int see1 = p.causal ? min(pos, t_end - 1) : t_end - 1;
          const int see0 = p.window > 0 ? pos - p.window + 1 : 0;
          const float x =
              t <= see1 && t >= see0 ? s_s[r * (kStep + 1) + lane] * s_c[r] : -INFINITY;
          float mx = x;
#pragma unroll
          for (int e = 16; e > 0; e >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, e));
          const float mn = fmaxf(m[i], mx);
          f = m[i] == mn ? 1.0f : ex2(m[i] - mn);
          m[i] = mn;
          y = ex2(x + (mn == -INFINITY ? 0.0f : kUp - mn));
          l[i] = fmaf(l[i], f, y);
        }
        s_p[r * (kStep + 8) + lane] = __float2half_rn(y);
        float sum = l[i];
        if (last) {
#pragma unroll
          for (int e = 16; e > 0; e >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, e);
        }
        if (lane == 0) {
          s_f[r] = f;
          if (last) {
            s_m[r] = m[i] == -INFINITY ? -INFINITY : m[i] - kUp;
            s_l[r] = sum;
          }
        }
      }
      __syncthreads();
      // ---- O += P V: the warp's columns
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float f0 = s_f[mt * 16 + (lane >> 2)], f1 = s_f[mt * 16 + 8 + (lane >> 2)];
        uint32_t a0[4], a1[4];
        ldsm4(a0, s_p + (mt * 16 + (lane & 15)) * (kStep + 8) + (lane >> 4) * 8);
        ldsm4(a1, s_p + (mt * 16 + (lane & 15)) * (kStep + 8) + 16 + (lane >> 4) * 8);
#pragma unroll
        for (int k = 0; k < kNT; ++k) {
          uint32_t vv[4];
          ldsm4_t(vv, s_v[buf] + lane * kPitch + (warp * kNT + k) * 8);
          float* c = o[mt][k];
          c[0] *= f0;
          c[1] *= f0;
          c[2] *= f1;
          c[3] *= f1;
          mma16(o[mt][k], a0, vv[0], vv[1]);
          mma16(o[mt][k], a1, vv[2], vv[3]);
        }
      }
      buf ^= 1;
      if (last) break;
    }

    // ---- out
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = mt * 16 + half * 8 + (lane >> 2);
        if (r >= rows) continue;
        const float ls = s_l[r];
        const int tok = r / p.g;
        const int64_t row = (int64_t)(row0 + tok) * p.Hq + h * p.g + (r - tok * p.g);
        const float inv = ls > 0.0f || ls != ls ? 1.0f / ls : 0.0f;
#pragma unroll
        for (int k = 0; k < kNT; ++k) {
          const int dim = (warp * kNT + k) * 8 + (lane & 3) * 2;
          const float x0 = o[mt][k][2 * half], x1 = o[mt][k][2 * half + 1];
          if (slot >= 0)
            *reinterpret_cast<float2*>(p.part_o + ((int64_t)slot * kR + r) * D + dim) =
                make_float2(x0, x1);
          else
            *reinterpret_cast<__nv_bfloat162*>(p.out + row * D + dim) =
                __floats2bfloat162_rn(x0 * inv, x1 * inv);
        }
        if (warp == 0 && (lane & 3) == 0) {
          if (slot >= 0)
            p.part_ml[(int64_t)slot * kR + r] = make_float2(s_m[r], ls);
          else if (p.lse != nullptr)
            p.lse[row] = ls > 0.0f || ls != ls ? (s_m[r] + log2f(ls)) * 0.69314718f : -INFINITY;
        }
      }
  }
}

// Joins the partial sums of contexts in several parts, in the parts' order.  A
// block takes every gridDim.y-th row; of few parts all its rows at once, of
// many (a head's context of 8192 tokens has 296) one after the other, with
// more warps to share the parts.  A lane takes D / 32 dims.
template <int D, int MT>
__global__ void __launch_bounds__(kDirThreads) chunk_direct_join_kernel(ChunkParams p) {
  constexpr int kR = MT * 16, E = D / 32, kMost = (kR + kJoinRows - 1) / kJoinRows, kPre = 4;
  __shared__ float s_o[kDirWarps][D];
  __shared__ float s_w[kMost][kMaxParts];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Split c = reinterpret_cast<const Split*>(p.cuts)[blockIdx.x];
  if ((int)blockIdx.x >= p.plan[0].npair) return;   // (what is read there is not used)
  const int parts = c.parts;
  const int y = (int)blockIdx.y, dy = (int)gridDim.y;
  if (y >= c.rows) return;
  const int mine = (c.rows - y + dy - 1) / dy;   // rows of the block
  const int at_once = parts > 32 ? 1 : mine > 2 ? min(4, kMost) : mine;
  const int i = warp % at_once, grp = warp / at_once, groups = kDirWarps / at_once;
#pragma unroll 1
  for (int i0 = 0; i0 < mine; i0 += at_once) {
    const int r = y + (i0 + i) * dy;
    const bool live = i0 + i < mine;
    auto at = [&](int s) { return (int64_t)(c.slot + s) * kR + r; };
    float m = -INFINITY, z = 0.0f, o[E] = {};
    if (live) {
      // the warp's first sums are on their way while the weights are found
      float x[kPre][E];
#pragma unroll
      for (int j = 0; j < kPre; ++j)
        if (grp + j * groups < parts)
#pragma unroll
          for (int k = 0; k < E; ++k)
            x[j][k] = p.part_o[at(grp + j * groups) * D + lane * E + k];
      // every warp of the row finds the weights (the same ones)
      float* w = s_w[i];
#pragma unroll 1
      for (int s = lane; s < parts; s += 32) m = fmaxf(m, p.part_ml[at(s)].x);
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, e));
#pragma unroll 1
      for (int s = lane; s < parts; s += 32) {
        const float2 ml = p.part_ml[at(s)];
        // what saw nothing has no weight (its sums are zero)
        const float f = ml.x == -INFINITY && ml.y == 0.0f ? 0.0f : ex2(ml.x - m);
        w[s] = f;
        z = fmaf(ml.y, f, z);
      }
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) z += __shfl_xor_sync(0xffffffffu, z, e);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kPre; ++j)
        if (grp + j * groups < parts)
#pragma unroll
          for (int k = 0; k < E; ++k) o[k] = fmaf(x[j][k], w[grp + j * groups], o[k]);
#pragma unroll 8
      for (int s = grp + kPre * groups; s < parts; s += groups) {
        const float f = w[s];
        const float* src = p.part_o + at(s) * D + lane * E;
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] = fmaf(src[k], f, o[k]);
      }
#pragma unroll
      for (int k = 0; k < E; ++k) s_o[warp][lane * E + k] = o[k];
    }
    __syncthreads();
    if (live && grp == 0) {
      for (int k = 1; k < groups; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += s_o[warp + k * at_once][lane * E + e];
      const int tok = r / p.g;
      const int64_t row = (int64_t)(c.row0 + tok) * p.Hq + c.h * p.g + (r - tok * p.g);
      const float inv = z > 0.0f || z != z ? 1.0f / z : 0.0f;
#pragma unroll
      for (int k = 0; k < E; k += 2)
        *reinterpret_cast<__nv_bfloat162*>(p.out + row * D + lane * E + k) =
            __floats2bfloat162_rn(o[k] * inv, o[k + 1] * inv);
      if (p.lse != nullptr && lane == 0)
        p.lse[row] = z > 0.0f || z != z ? (m + log2f(z)) * 0.69314718f : -INFINITY;
    }
    __syncthreads();
  }
}

// At most a thread per request, 32 rows per request and KV head, and counts
// of units that fit 32 bits.
bool direct_fits(int B, int64_t n_tok, int g, int max_q, int max_len) {
  const int64_t q = max_q < n_tok ? max_q : n_tok;
  return B <= kDirThreads && q * g <= 32 && max_len <= 1 << 20;
}

size_t direct_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int max_q, int max_len,
                              int64_t total_len) {
  const int64_t q = max_q < n_tok ? max_q : n_tok;
  return direct_layout(pad_rows(q * (Hq / Hkv)), d, direct_ctas(B, Hkv, max_len, total_len)).total;
}

template <int D, int MT>
static sdk_status launch_direct_d(const ChunkParams& p, cudaStream_t stream) {
  chunk_direct_kernel<D, MT><<<(unsigned)p.ctas, kDirThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SDK_ERR_CUDA;
  // contexts in several parts: half as many as parts
  const int rows = p.max_q * p.g, most = min(p.ctas, p.B * p.Hkv);
  const int y = min(rows, max(kJoinRows, 4 * num_sms() / most));
  if (p.ctas > 1 && launch_after(chunk_direct_join_kernel<D, MT>, dim3((unsigned)most, (unsigned)y),
                                 kDirThreads, 0, stream, p) != cudaSuccess)
    return SDK_ERR_CUDA;
  return SDK_OK;
}

sdk_status launch_chunk_direct(ChunkParams p, int64_t total_len, char* workspace,
                               cudaStream_t stream) {
  const int rows = pad_rows((int64_t)p.max_q * p.g);
  p.ctas = direct_ctas(p.B, p.Hkv, p.max_len, total_len);
  const DirectLayout l = direct_layout(rows, p.d, p.ctas);
  p.cuts = workspace + l.splits;
  p.part_ml = reinterpret_cast<float2*>(workspace + l.ml);
  p.part_o = reinterpret_cast<float*>(workspace + l.po);
  if (p.d == 128) return rows > 16 ? launch_direct_d<128, 2>(p, stream) : launch_direct_d<128, 1>(p, stream);
  return rows > 16 ? launch_direct_d<64, 2>(p, stream) : launch_direct_d<64, 1>(p, stream);
}

}  // namespace sdk
