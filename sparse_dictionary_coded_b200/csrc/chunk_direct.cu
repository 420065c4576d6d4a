// Chunk attention (sdk_chunk_attn) for few rows over short contexts, in one
// pass: a CTA rebuilds 32 tokens' keys and values
//   K_t = sum_j c_tj D_K[i_tj],  V_t = sum_j c_tj D_V[i_tj]
// as fp16 in shared memory and attends to them at once, with a running
// maximum and sum per row, so that nothing but the partial sums of contexts
// that several CTAs share goes through the workspace.
//   chunk_direct_kernel       shares of all contexts
//   chunk_direct_join_kernel  the sums of contexts that several shares hold
// What counts here is the chain of dependent loads: lengths, page, code words,
// atoms' rows (16 in flight a lane).
#include "chunk_plan.cuh"
#include "tc_ptx.cuh"

namespace sdk {

namespace {

constexpr int kDirThreads = 256, kDirWarps = kDirThreads / 32;
constexpr int kUnit = 16;          // tokens of a unit of work
constexpr int kStep = 32;          // tokens rebuilt and attended to at a time
constexpr int kJoinGroups = 4;     // warps that share a row's parts when joining
constexpr float kUp = 14.0f;       // log2 of P's offset: its smallest fp16 step is 2^-38 of the largest term

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// What share c of the work starts with, left for the join.
struct Cut {
  int64_t u0;          // its first unit
  int64_t lo, hi;      // the units of the context that unit belongs to
  int row0, rows, h;
};

struct DirectLayout {
  size_t cuts, ml, po, total;
};

DirectLayout direct_layout(int B, int rows, int d, int ctas) {
  DirectLayout l;
  l.cuts = up256(sizeof(WsHeader) + sizeof(ReqPlan));
  l.ml = up256(l.cuts + (size_t)ctas * sizeof(Cut));
  l.po = up256(l.ml + (size_t)2 * ctas * rows * 8);
  l.total = up256(l.po + (size_t)2 * ctas * rows * d * 4);
  return l;
}

int pad_rows(int64_t rows) { return rows <= 16 ? 16 : 32; }

// Shares at most: two CTAs per SM, or one for every unit there can be.
int direct_ctas(int B, int Hkv, int max_len, int64_t total_len) {
  int64_t units = (int64_t)B * (max_len / kUnit + 2);
  if (total_len > 0 && total_len / kUnit + 2 * (int64_t)B < units) units = total_len / kUnit + 2 * (int64_t)B;
  units *= Hkv;
  return (int)(units < 2 * num_sms() ? units : 2 * num_sms());
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

// Every CTA scans the requests itself (at most one per thread) and takes an
// equal share of the units of 16 tokens of all (request, KV head) contexts, in
// that order; a share's segments are attended to one after the other.  The
// products are small (32 tokens and 16 or 32 rows at a time), so the warps'
// own matrix instructions do them; P and the sums as in chunk_attn.cu.
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
  __shared__ int64_t s_work[kDirThreads + 1];
  __shared__ int4 s_req[kDirThreads];             // row0, n, len, first token
  __shared__ int64_t s_warp[32];
  __shared__ int s_units;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch();

  // ---- the plan.  Tiles of 128 tokens are what the caller's bound on the
  // lengths is held against, as in the other form.
  if (tid == 0) {
    s_units = 0;
    s_work[0] = 0;
  }
  unsigned err = 0;
  ReqPlan rq = {};
  int units = 0;
  if (tid < p.B) {
    rq = check_request(p, tid, &err);
    if (rq.n > 0) {
      // the first token any row sees, rounded down to a unit
      const int seen = p.window > 0 ? max(rq.len - rq.n - p.window + 1, 0) : 0;
      rq.lo = min(seen, rq.len) / kUnit * kUnit;
      units = max((rq.len - rq.lo + kUnit - 1) / kUnit, 1);
    }
  }
  int64_t both;
  const int64_t upto =
      block_scan64(((int64_t)rq.ntiles << 32) + units, s_warp, &both);
  if (tid < p.B) {
    if (rq.n > 0 && (upto >> 32) > p.cap_tiles) {
      err = SDK_ERR_CAPACITY;
      rq.n = 0;
    } else if (units > 0) {
      atomicMax(&s_units, (int)(uint32_t)upto);
    }
    s_work[tid + 1] = (int64_t)(uint32_t)upto * p.Hkv;
    s_req[tid] = make_int4(rq.row0, rq.n, rq.len, rq.lo);
    if (err && blockIdx.x == 0) record_error(p.hdr, err, 0x75000000u | (uint32_t)tid);
  }
  __syncthreads();
  const int64_t U = (int64_t)s_units * p.Hkv;
  const int N = (int)min(U, (int64_t)gridDim.x), me = (int)blockIdx.x;
  if (me == 0 && tid == 0) {
    p.plan[0].work0 = U;
    p.plan[0].npair = N;
  }
  if (me >= N) return;
  int64_t u = U * me / N;
  const int64_t u_end = U * (me + 1) / N;
  int b = 0;
  {
    int hi = p.B;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (s_work[mid] <= u) b = mid; else hi = mid;
    }
  }

  const int rec = lane / LPR, sub = lane % LPR, kv = rec & 1;
  const uint4* dict = reinterpret_cast<const uint4*>(kv ? p.dv : p.dk);
  int buf = 0;
#pragma unroll 1
  for (bool first = true; u < u_end; first = false) {
    while (s_work[b + 1] <= u) ++b;
    const int4 r4 = s_req[b];
    const int row0 = r4.x, n = r4.y, len = r4.z, rows = n * p.g;
    const int64_t w0 = s_work[b];
    const int per = (int)((uint32_t)((s_work[b + 1] - w0) / p.Hkv));
    const int rel = (int)(u - w0), h = rel / per, ui = rel - h * per;
    const int cnt = (int)min((int64_t)(per - ui), u_end - u);
    const int t_begin = r4.w + ui * kUnit, t_end = min(len, t_begin + cnt * kUnit);
    // partial sums: of the share's first segment or of its last
    const int slot = cnt < per ? 2 * me + (first ? 0 : 1) : -1;
    if (first && tid == 0) {
      Cut cut;
      cut.u0 = u;
      cut.lo = u - ui;
      cut.hi = cut.lo + per;
      cut.row0 = row0;
      cut.rows = rows;
      cut.h = h;
      reinterpret_cast<Cut*>(p.cuts)[me] = cut;
    }
    // code words of the step at t0: the warp's tokens t0 + warp TPS, and so on
    uint32_t w[NU][WPL];
    auto load_words = [&](int t0) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int t = t0 + (i * kDirWarps + warp) * TPS + (rec >> 1);
#pragma unroll
        for (int k = 0; k < WPL; ++k) w[i][k] = 0u;
        if (t < t_end) {
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
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int r = (i * kDirWarps + warp) * TPS + (rec >> 1);
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (t0 + r - (rec >> 1) < t_end) {
          bool bad = false;
          y = rebuild_piece<D, true>(p, dict, w[i], rec, sub, &bad);
          if (bad) record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x77000000u | (uint32_t)b);
        }
        *reinterpret_cast<uint4*>((kv ? s_v[buf] : s_k) + r * kPitch + sub * 8) = y;
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
    u += cnt;
  }
}

// Joins the partial sums of the contexts that several shares hold, in the
// shares' order: share c stands for the context that its first unit lies
// inside of, if that is the first cut there.  Four warps share a row's parts,
// a lane takes D / 32 dims.
template <int D, int MT>
__global__ void __launch_bounds__(kDirThreads) chunk_direct_join_kernel(ChunkParams p) {
  constexpr int kR = MT * 16, E = D / 32, kRowsBlock = kDirWarps / kJoinGroups;
  __shared__ float s_o[kDirWarps][D];
  pdl_wait();
  const Cut* cuts = reinterpret_cast<const Cut*>(p.cuts);
  const int c = (int)blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Cut cut = cuts[c];                         // (of a share that is not there: not used)
  const int64_t before = cuts[c - 1].u0, U = p.plan[0].work0;
  const int shares = p.plan[0].npair;
  if (c >= shares || cut.u0 == cut.lo || before > cut.lo) return;   // no cut, or an earlier one
  if ((int)blockIdx.y * kRowsBlock >= cut.rows) return;
  const int grp = warp % kJoinGroups, r = blockIdx.y * kRowsBlock + warp / kJoinGroups;
  const bool live = r < cut.rows;
  // share c - 1 ends with its part, the shares c .. last start with theirs
  const int slot0 = 2 * (c - 1) + (before < cut.lo ? 1 : 0);
  const int last = (int)((cut.hi * shares - 1) / U), parts = last - c + 2;
  auto at = [&](int s) { return (int64_t)(s == 0 ? slot0 : 2 * (c - 1 + s)) * kR + r; };
  float m = -INFINITY, z = 0.0f, o[E] = {};
  if (live) {
    for (int s = lane; s < parts; s += 32) m = fmaxf(m, p.part_ml[at(s)].x);
#pragma unroll
    for (int e = 16; e > 0; e >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, e));
    // what saw nothing has no weight (its sums are zero)
    auto weight = [&](const float2& ml) { return ml.x == -INFINITY && ml.y == 0.0f ? 0.0f : ex2(ml.x - m); };
    for (int s = lane; s < parts; s += 32) {
      const float2 ml = p.part_ml[at(s)];
      z = fmaf(ml.y, weight(ml), z);
    }
#pragma unroll
    for (int e = 16; e > 0; e >>= 1) z += __shfl_xor_sync(0xffffffffu, z, e);
#pragma unroll 4
    for (int s = grp; s < parts; s += kJoinGroups) {
      const float f = weight(p.part_ml[at(s)]);
      const float* src = p.part_o + at(s) * D + lane * E;
#pragma unroll
      for (int k = 0; k < E; ++k) o[k] = fmaf(src[k], f, o[k]);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) s_o[warp][lane * E + k] = o[k];
  }
  __syncthreads();
  if (!live || grp > 0) return;
#pragma unroll
  for (int i = 1; i < kJoinGroups; ++i)
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] += s_o[warp + i][lane * E + k];
  const int tok = r / p.g;
  const int64_t row = (int64_t)(cut.row0 + tok) * p.Hq + cut.h * p.g + (r - tok * p.g);
  const float inv = z > 0.0f || z != z ? 1.0f / z : 0.0f;
#pragma unroll
  for (int k = 0; k < E; k += 2)
    *reinterpret_cast<__nv_bfloat162*>(p.out + row * D + lane * E + k) =
        __floats2bfloat162_rn(o[k] * inv, o[k + 1] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = z > 0.0f || z != z ? (m + log2f(z)) * 0.69314718f : -INFINITY;
}

// At most a thread per request, 32 rows per request and KV head, and counts
// of units that fit 32 bits.
bool direct_fits(int B, int64_t n_tok, int g, int Hkv, int max_q, int max_len) {
  const int64_t q = max_q < n_tok ? max_q : n_tok;
  return B <= kDirThreads && q * g <= 32 && max_len <= 1 << 20 && (int64_t)Hkv * max_len <= 1 << 30;
}

size_t direct_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int max_q, int max_len,
                              int64_t total_len) {
  const int64_t q = max_q < n_tok ? max_q : n_tok;
  return direct_layout(B, pad_rows(q * (Hq / Hkv)), d, direct_ctas(B, Hkv, max_len, total_len)).total;
}

template <int D, int MT>
static sdk_status launch_direct_d(const ChunkParams& p, cudaStream_t stream) {
  chunk_direct_kernel<D, MT><<<(unsigned)p.ctas, kDirThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SDK_ERR_CUDA;
  const int rows = p.max_q * p.g, each = kDirWarps / kJoinGroups;
  if (p.ctas > 1 &&
      launch_after(chunk_direct_join_kernel<D, MT>,
                   dim3((unsigned)(p.ctas - 1), (unsigned)((rows + each - 1) / each)), kDirThreads, 0,
                   stream, p) != cudaSuccess)
    return SDK_ERR_CUDA;
  return SDK_OK;
}

sdk_status launch_chunk_direct(ChunkParams p, int64_t total_len, char* workspace,
                               cudaStream_t stream) {
  const int rows = pad_rows((int64_t)p.max_q * p.g);
  p.ctas = direct_ctas(p.B, p.Hkv, p.max_len, total_len);
  const DirectLayout l = direct_layout(p.B, rows, p.d, p.ctas);
  p.cuts = workspace + l.cuts;
  p.part_ml = reinterpret_cast<float2*>(workspace + l.ml);
  p.part_o = reinterpret_cast<float*>(workspace + l.po);
  if (p.d == 128) return rows > 16 ? launch_direct_d<128, 2>(p, stream) : launch_direct_d<128, 1>(p, stream);
  return rows > 16 ? launch_direct_d<64, 2>(p, stream) : launch_direct_d<64, 1>(p, stream);
}

}  // namespace sdk
