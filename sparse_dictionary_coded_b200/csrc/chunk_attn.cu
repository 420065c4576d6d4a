// Attention of new tokens over paged codes (sdk_chunk_attn, include/sdk.h).
//
// Two kernels: rebuild_kernel writes the context's vectors
//   K_t = sum_j c_tj D_K[i_tj],  V_t = sum_j c_tj D_V[i_tj]
// once per call as fp16 tiles of 128 tokens in the workspace, and
// chunk_attn_kernel computes softmax(scale q K^T) V over the tiles.
#include "paged.cuh"

namespace sdk {

namespace {

constexpr int kTile = 128;        // tokens of a rebuilt tile
constexpr int kRebThreads = 256;
constexpr int kRebTok = 32;       // tokens of one work item of rebuild_kernel

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct ChunkLayout {
  size_t plan, kt, vt, total;
};

ChunkLayout chunk_layout(int B, int Hkv, int d, int64_t cap_tiles) {
  ChunkLayout l;
  const size_t tiles = (size_t)cap_tiles * Hkv * kTile * d * 2;
  l.plan = sizeof(WsHeader);
  l.kt = up256(l.plan + (size_t)B * sizeof(ReqPlan));
  l.vt = l.kt + tiles;
  l.total = l.vt + tiles;
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
// workspace for the attention kernel.  A work item is 32 tokens of one KV
// head; D / 8 lanes rebuild one vector (16-byte pieces of an atom's row), a
// warp a token's key and value (two tokens at head_dim 64).  Bound by the
// gathers of 2 x 16 atom rows (8 KB per token and head at head_dim 128)
// from L2.
template <int D>
__global__ void __launch_bounds__(kRebThreads) rebuild_kernel(ChunkParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_tile0 = sm;              // [B + 1]
  int32_t* s_lo = s_tile0 + p.B + 1;  // [B]
  int32_t* s_len = s_lo + p.B;        // [B]
  __shared__ uint32_t s_warp[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t base = 0;
  if (tid == 0) s_tile0[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += kRebThreads) {
    const int b = b0 + tid;
    int row0 = 0, n = 0, len = 0, lo = 0;
    uint32_t nt = 0, err = 0;
    if (b < p.B) {
      row0 = p.cu_q[b];
      const int row1 = p.cu_q[b + 1];
      len = p.lens[b];
      if (row0 < 0 || row1 < row0 || row1 > p.n_tok || len < 0) {
        err = SDK_ERR_DEVICE_CHECK;
      } else if (row1 - row0 > p.max_q || len > p.max_len) {
        err = SDK_ERR_CAPACITY;
      } else {
        n = row1 - row0;
      }
      if (n > 0) {
        // the first row's position len - n sees tokens from len - n - window + 1 on
        if (p.window > 0) lo = max(0, (int)max((int64_t)len - n - p.window + 1, (int64_t)0));
        lo = lo / kTile * kTile;
        nt = (uint32_t)((max(len - lo, 0) + kTile - 1) / kTile);
      }
    }
    uint32_t total;
    const uint32_t upto = base + block_incl_scan(nt, s_warp, &total);
    if (b < p.B) {
      if (upto > (uint32_t)p.cap_tiles && nt > 0) {   // total_len does not hold
        err = SDK_ERR_CAPACITY;
        n = 0;
      }
      s_tile0[b + 1] = (int)min(upto, (uint32_t)p.cap_tiles);
      s_lo[b] = lo;
      s_len[b] = n > 0 ? len : 0;
      if (blockIdx.x == 0) {
        ReqPlan r;
        r.row0 = row0;
        r.n = n;
        r.len = len;
        r.lo = lo;
        r.tile0 = (int)(upto - nt);
        r.ntiles = n > 0 ? (int)nt : 0;
        r.pad[0] = r.pad[1] = 0;
        p.plan[b] = r;
        if (err) record_error(p.hdr, err, 0x75000000u | (uint32_t)b);
      }
    }
    base += total;
  }
  __syncthreads();

  constexpr int LPR = D / 8;           // lanes per record
  constexpr int TPS = 32 / (2 * LPR);  // tokens a warp rebuilds at a time
  constexpr int WPL = 16 / LPR;        // code words a lane holds
  constexpr int kTokWarp = kRebTok / (kRebThreads / 32);
  const int rec = lane / LPR, sub = lane % LPR;
  const int kv = rec & 1;
  const uint4* dict = reinterpret_cast<const uint4*>(kv ? p.dv : p.dk);
  char* tiles = reinterpret_cast<char*>(kv ? p.vt : p.kt);
  const int64_t items = (int64_t)s_tile0[p.B] * p.Hkv * (kTile / kRebTok);
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int part = (int)(it % (kTile / kRebTok));
    const int64_t th = it / (kTile / kRebTok);
    const int h = (int)(th % p.Hkv);
    const int tile = (int)(th / p.Hkv);
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_tile0[mid] <= tile) lo = mid; else hi = mid;
    }
    const int b = lo;
    char* dst = tiles + ((int64_t)tile * p.Hkv + h) * (kTile * D * 2);
#pragma unroll 1
    for (int u = 0; u < kTokWarp; u += TPS) {
      const int r = part * kRebTok + warp * kTokWarp + u + (rec >> 1);   // row of the tile
      const int t = s_lo[b] + (tile - s_tile0[b]) * kTile + r;
      uint32_t w[WPL];
#pragma unroll
      for (int i = 0; i < WPL; ++i) w[i] = 0u;
      if (t < s_len[b]) {
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
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      bool bad = false;
#pragma unroll
      for (int j = 0; j < kAtoms; ++j) {
        const uint32_t x = __shfl_sync(0xffffffffu, w[j % WPL], rec * LPR + j / WPL);
        uint32_t a = word_idx(x);
        float c = word_coef(x);
        if (a >= (uint32_t)p.n) {
          bad = true;
          a = 0;
          c = 0.0f;
        }
        const uint4 v = __ldg(dict + (int64_t)a * LPR + sub);
        acc[0] = fmaf(c, bf16_lo(v.x), acc[0]);
        acc[1] = fmaf(c, bf16_hi(v.x), acc[1]);
        acc[2] = fmaf(c, bf16_lo(v.y), acc[2]);
        acc[3] = fmaf(c, bf16_hi(v.y), acc[3]);
        acc[4] = fmaf(c, bf16_lo(v.z), acc[4]);
        acc[5] = fmaf(c, bf16_hi(v.z), acc[5]);
        acc[6] = fmaf(c, bf16_lo(v.w), acc[6]);
        acc[7] = fmaf(c, bf16_hi(v.w), acc[7]);
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

// One warp per (row, query head): lanes hold D / 32 dims, one pass over the
// tokens with the running maximum and sum.
template <int D>
__global__ void __launch_bounds__(128) chunk_attn_kernel(ChunkParams p) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ReqPlan rp = p.plan[blockIdx.y];
  const int64_t e = (int64_t)blockIdx.x * 4 + warp;
  const int i = (int)(e / p.Hq), hq = (int)(e % p.Hq);
  if (i >= rp.n) return;
  const int h = hq / p.g;
  const int64_t row = (int64_t)(rp.row0 + i) * p.Hq + hq;
  float q[E], o[E];
#pragma unroll
  for (int k = 0; k < E; ++k) {
    q[k] = __uint_as_float((uint32_t)p.q[row * D + lane * E + k] << 16);
    o[k] = 0.0f;
  }
  const int pos = rp.len - rp.n + i;
  const int t1 = p.causal ? min(pos + 1, rp.len) : rp.len;
  const int t0 = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float m = -INFINITY, z = 0.0f;
  for (int t = t0; t < t1; ++t) {
    const int tl = (t - rp.lo) / kTile, r = (t - rp.lo) % kTile;
    const int64_t base = ((int64_t)(rp.tile0 + tl) * p.Hkv + h) * (kTile * D * 2);
    const int off = tile_off(r, lane * E / 8) + (lane * E % 8) * 2;
    const __half* kp = reinterpret_cast<const __half*>(reinterpret_cast<const char*>(p.kt) + base + off);
    const __half* vp = reinterpret_cast<const __half*>(reinterpret_cast<const char*>(p.vt) + base + off);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < E; ++k) s = fmaf(q[k], __half2float(kp[k]), s);
    s = warp_sum(s) * p.scale;
    const float mn = fmaxf(m, s), a = __expf(m - mn), x = __expf(s - mn);
    z = z * a + x;
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = fmaf(x, __half2float(vp[k]), o[k] * a);
    m = mn;
  }
#pragma unroll
  for (int k = 0; k < E; ++k)
    p.out[row * D + lane * E + k] =
        __bfloat16_as_ushort(__float2bfloat16_rn(z > 0.0f || z != z ? o[k] / z : 0.0f));
  if (p.lse != nullptr && lane == 0) p.lse[row] = m + logf(z);
}

int64_t chunk_cap_tiles(int B, int max_len, int64_t total_len) {
  const int64_t each = (int64_t)B * ((max_len + (int64_t)kTile - 1) / kTile);
  if (total_len <= 0) return each;
  const int64_t sum = total_len / kTile + B;   // every context ends inside a tile at most once
  return sum < each ? sum : each;
}

size_t chunk_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q,
                             int max_len, int64_t total_len) {
  return chunk_layout(B, Hkv, d, chunk_cap_tiles(B, max_len, total_len)).total;
}

template <int D>
static sdk_status launch_d(const ChunkParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)(3 * p.B + 1) * 4;
  static unsigned long long attr_set = 0ull;
  if (device_needs_setup(&attr_set)) {
    if (cudaFuncSetAttribute(rebuild_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (3 * SDK_MAX_REQUESTS + 1) * 4) != cudaSuccess)
      return SDK_ERR_CUDA;
    device_setup_done(&attr_set);
  }
  int64_t grid = (int64_t)p.cap_tiles * p.Hkv * (kTile / kRebTok);
  if (grid > 8 * num_sms()) grid = 8 * num_sms();
  rebuild_kernel<D><<<(unsigned)grid, kRebThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SDK_ERR_CUDA;
  const int64_t gx = ((int64_t)p.max_q * p.Hq + 3) / 4;
  chunk_attn_kernel<D><<<dim3((unsigned)gx, (unsigned)p.B), 128, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SDK_OK : SDK_ERR_CUDA;
}

sdk_status launch_chunk_attn(ChunkParams p, char* workspace, cudaStream_t stream) {
  const ChunkLayout l = chunk_layout(p.B, p.Hkv, p.d, p.cap_tiles);
  p.hdr = reinterpret_cast<WsHeader*>(workspace);
  p.plan = reinterpret_cast<ReqPlan*>(workspace + l.plan);
  p.kt = reinterpret_cast<__half*>(workspace + l.kt);
  p.vt = reinterpret_cast<__half*>(workspace + l.vt);
  return p.d == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace sdk
