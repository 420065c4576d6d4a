// The paged code store: plans of a step (sdk_block_tables) and the writes
// of code words to their slots (sdk_paged_store).  The operations are
// defined in include/sdk.h.
#include "paged.cuh"

namespace sdk {

namespace {

constexpr uint32_t kCap = 0x7FFFFFFFu;   // sums saturate here (a + b fits 32 bits)

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kCap); }

// Inclusive saturating scan of one value (<= kCap) per thread of a block of T.
template <int T>
__device__ __forceinline__ uint32_t block_sat_scan(uint32_t v, uint32_t* s_warp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = sat_add(v, t);
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    uint32_t t = lane < T / 32 ? s_warp[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t = sat_add(t, u);
    }
    if (lane < T / 32) s_warp[lane] = t;
  }
  __syncthreads();
  const uint32_t r = warp > 0 ? sat_add(v, s_warp[warp - 1]) : v;
  *total = s_warp[T / 32 - 1];
  __syncthreads();
  return r;
}

}  // namespace

// One step's plan.  Every CTA scans the requests itself (rows, then pages:
// two scans of at most 4096 values in shared memory cost a few hundred ns, a
// second launch or a grid-wide wait would cost more), then takes its share
// of the table entries and of the slots by binary search in the scans; of many
// rows a thread takes four neighbours.  The page of a slot comes from the free stack when
// this call assigns it, so no CTA reads an entry another one writes.  Bound
// by its launch and the chain load - scan - load for a step of single tokens
// (2.6 us for 4 requests in a graph), for prompts too (64 of up to 16384 tokens:
// 4.7 us; four rows far apart, a search each: 6.4 us).
// T threads: 256 for up to 256 requests, else 1024.
template <int T>
__global__ void __launch_bounds__(T) block_tables_kernel(TableParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_row = sm;                  // [B + 1] first row of every request
  int32_t* s_fresh = s_row + p.B + 1;   // [B + 1] pages taken before it
  int32_t* s_len = s_fresh + p.B + 1;   // [B] its length, -1: refused
  __shared__ uint32_t s_warp[32];
  const int tid = threadIdx.x;
  const uint32_t P = (uint32_t)p.page_size;
  int n_free = *p.n_free;
  int len0 = 0, n0 = 0;                 // the first requests', loaded beside it
  if (tid < p.B) {
    len0 = p.lens[tid];
    n0 = p.n_new[tid];
  }
  if (n_free < 0 || n_free > p.n_stack) {
    if (tid == 0 && blockIdx.x == 0) record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x70000001u);
    n_free = min(max(n_free, 0), p.n_stack);
  }
  if (tid == 0) s_row[0] = s_fresh[0] = 0;
  uint32_t row0 = 0, page0 = 0;
  for (int b0 = 0; b0 < p.B; b0 += T) {
    const int b = b0 + tid;
    int len = len0, n = n0;
    if (b0 > 0 && b < p.B) {
      len = p.lens[b];
      n = p.n_new[b];
    }
    if (b >= p.B) len = n = 0;
    uint32_t rows, pages;
    const uint32_t row1 = sat_add(row0, block_sat_scan<T>((uint32_t)max(n, 0), s_warp, &rows));
    // refused: 1 a bound or the pool, 2 a bad length
    int refused = 0;
    uint32_t need = 0, have = 0;
    if (len < 0 || n < 0 || (int64_t)len + n > 0x7FFFFFFF) {
      refused = 2;
    } else {
      have = ((uint32_t)len + P - 1) / P;
      const uint32_t want = ((uint32_t)len + (uint32_t)n + P - 1) / P;
      if (want > (uint32_t)p.max_pages || (n > 0 && row1 > (uint32_t)p.max_new))
        refused = 1;
      else
        need = want - have;
    }
    const uint32_t upto = sat_add(page0, block_sat_scan<T>(need, s_warp, &pages));
    if (!refused && upto > (uint32_t)n_free && need > 0) refused = 1;
    if (b < p.B) {
      s_row[b + 1] = (int)min(row1, (uint32_t)p.max_new);
      // the pages really taken: a refused request and all that follow it and
      // need pages stop the count, since `upto` only grows
      s_fresh[b + 1] = (int)(upto > (uint32_t)n_free ? 0xFFFFFFFFu : upto);
      s_len[b] = refused ? -1 : len;
      if (blockIdx.x == 0) {
        p.new_lens[b] = refused ? len : len + n;
        if (refused)
          record_error(p.hdr, refused == 2 ? SDK_ERR_DEVICE_CHECK : SDK_ERR_CAPACITY,
                       0x71000000u | (uint32_t)b);
      }
    }
    row0 = sat_add(row0, rows);
    page0 = sat_add(page0, pages);
  }
  __syncthreads();
  int taken = (int)page0;
  if (page0 > (uint32_t)n_free) {
    // s_fresh of a request behind the one that did not fit: the pages taken
    // before it are those of the last request that fitted
    __shared__ int s_taken;
    if (tid == 0) s_taken = 0;
    __syncthreads();
    int m = 0;
    for (int b = tid; b < p.B; b += T) m = max(m, s_fresh[b + 1]);
    m = (int)__reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0 && m > 0) atomicMax(&s_taken, m);
    __syncthreads();
    taken = s_taken;
    for (int b = tid; b < p.B; b += T)
      if (s_fresh[b + 1] < 0) s_fresh[b + 1] = taken;
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    for (int b = tid; b <= p.B; b += T) p.cu_new[b] = s_row[b];
    if (tid == 0) *p.n_free_out = n_free - taken;
  }
  const int64_t step = (int64_t)gridDim.x * T;
  const int64_t t0 = (int64_t)blockIdx.x * T + tid;
  auto fresh_page = [&](int e) {       // the e-th page taken
    const int pg = p.free_pages[n_free - 1 - e];
    if (pg >= 0 && pg < p.n_pages) return pg;
    record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x72000000u);
    return -1;
  };
  // the last b with first[b] <= e
  auto find = [&](const int32_t* first, int e) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= e) lo = mid; else hi = mid;
    }
    return lo;
  };
  for (int64_t e = t0; e < taken; e += step) {
    const int b = find(s_fresh, (int)e);
    const uint32_t have = ((uint32_t)s_len[b] + P - 1) / P;
    p.table[(int64_t)b * p.max_pages + have + ((int)e - s_fresh[b])] = fresh_page((int)e);
  }
  const int n_rows = s_row[p.B];
  // the page that holds token pos of request b, column col
  auto page_at = [&](int b, int len, uint32_t col, bool* fresh) {
    const uint32_t have = ((uint32_t)len + P - 1) / P;
    *fresh = col >= have;
    return *(*fresh ? p.free_pages + (n_free - 1 - (s_fresh[b] + (int)(col - have)))
                    : p.table + ((int64_t)b * p.max_pages + col));
  };
  auto slot_of = [&](int b, int pg, uint32_t off, bool fresh) {
    if (pg >= 0 && pg < p.n_pages) return (int64_t)pg * P + off;
    if (!fresh)                         // (a bad page of the stack is recorded above)
      record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x73000000u | (uint32_t)b);
    return (int64_t)-1;
  };
  constexpr int R = 4;                  // rows a thread has in flight
  if (p.max_new <= 2 * step) {
    for (int64_t r0 = t0; r0 < p.max_new; r0 += step) {
      int64_t slot = -1;
      if (r0 < n_rows) {
        const int b = find(s_row, (int)r0), len = s_len[b];
        if (len >= 0) {
          const uint32_t pos = (uint32_t)len + (uint32_t)((int)r0 - s_row[b]), col = pos / P;
          bool fresh;
          const int pg = page_at(b, len, col, &fresh);
          slot = slot_of(b, pg, pos - col * P, fresh);
        }
      }
      p.slot_map[r0] = slot;
    }
    return;
  }
  // many rows: four neighbours a thread, so that one search does for most
  const bool wide = ((uintptr_t)p.slot_map & 15) == 0;
  for (int64_t r0 = t0 * R; r0 < p.max_new; r0 += R * step) {
    int req[R], pg[R];
    uint32_t off[R];
    bool fresh[R];
    int b = r0 < n_rows ? find(s_row, (int)r0) : 0, len = s_len[b];
    uint32_t pos = (uint32_t)len + (uint32_t)((int)min(r0, (int64_t)n_rows) - s_row[b]), col = pos / P,
             o = pos - col * P;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t r = r0 + k;
      req[k] = -1;
      if (r < n_rows) {
        if (r >= s_row[b + 1]) {        // the next request with rows
          do ++b;
          while (r >= s_row[b + 1]);
          len = s_len[b];
          col = (uint32_t)len / P;
          o = (uint32_t)len - col * P;
        }
        if (len >= 0) {
          req[k] = b;
          off[k] = o;
          pg[k] = page_at(b, len, col, &fresh[k]);
        }
        if (++o == P) {
          o = 0;
          ++col;
        }
      }
    }
    int64_t slot[R];
#pragma unroll
    for (int k = 0; k < R; ++k)
      slot[k] = req[k] < 0 ? -1 : slot_of(req[k], pg[k], off[k], fresh[k]);
    if (wide && r0 + R <= p.max_new) {
      longlong2* dst = reinterpret_cast<longlong2*>(p.slot_map + r0);
      dst[0] = make_longlong2(slot[0], slot[1]);
      dst[1] = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (r0 + k < p.max_new) p.slot_map[r0 + k] = slot[k];
    }
  }
}

// Eight lanes copy one (token, KV head): four 16-byte pieces of key words,
// four of value words, to the 128-byte line of its slot.  Bound by HBM (the
// words are read once and written once): 16384 tokens of 8 heads, 33.7 MB, 8.2
// us, 5.2 in a graph.  One piece a thread: of four, all read before the first
// was written (10.2 us), of eight 15.8 us.  I: the type that counts the pieces.
template <typename I>
__global__ void __launch_bounds__(256) paged_store_kernel(StoreParams p) {
  const I items = (I)p.n_tok * (I)(p.Hkv * 8), step = (I)gridDim.x * 256;
  for (I e = (I)blockIdx.x * 256 + threadIdx.x; e < items; e += step) {
    const I rec = e >> 3, t = rec / (I)p.Hkv;
    const int c = (int)(e & 7), h = (int)(rec - t * (I)p.Hkv);
    const uint4 v =
        __ldg(reinterpret_cast<const uint4*>(c < 4 ? p.codes_k : p.codes_v) + rec * 4 + (c & 3));
    const int64_t slot = __ldg(p.slot_map + t);
    int64_t at = -1;                    // (one store at the end: both loads are issued first)
    if (slot >= (int64_t)p.n_pages * p.page_size) {
      record_error(p.hdr, SDK_ERR_DEVICE_CHECK, 0x74000000u);
    } else if (slot >= 0) {
      const uint32_t page = (uint32_t)slot / (uint32_t)p.page_size;
      const uint32_t off = (uint32_t)slot - page * (uint32_t)p.page_size;
      at = (((int64_t)page * p.Hkv + h) * p.page_size + off) * 8 + c;
    }
    if (at >= 0) reinterpret_cast<uint4*>(p.pages)[at] = v;
  }
}

template <int T>
static sdk_status launch_tables(const TableParams& p, cudaStream_t stream) {
  const int64_t work = p.max_new > p.B ? p.max_new : p.B;
  int64_t grid = (work + 4 * T - 1) / (4 * T);
  const int64_t most = (int64_t)num_sms() * (2048 / T);
  if (grid > most) grid = most;
  static unsigned long long attr_set = 0ull;
  if (device_needs_setup(&attr_set)) {
    if (cudaFuncSetAttribute(block_tables_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (3 * SDK_MAX_REQUESTS + 2) * 4) != cudaSuccess)
      return SDK_ERR_CUDA;
    device_setup_done(&attr_set);
  }
  block_tables_kernel<T><<<(unsigned)grid, T, (size_t)(3 * p.B + 2) * 4, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SDK_OK : SDK_ERR_CUDA;
}

sdk_status launch_block_tables(const TableParams& p, cudaStream_t stream) {
  return p.B <= 256 ? launch_tables<256>(p, stream) : launch_tables<1024>(p, stream);
}

sdk_status launch_paged_store(const StoreParams& p, cudaStream_t stream) {
  if (p.n_tok == 0) return SDK_OK;
  const int64_t items = p.n_tok * p.Hkv * 8;
  int64_t grid = (items + 255) / 256;
  if (grid > 128 * num_sms()) grid = 128 * num_sms();
  // an index and a step stay below 2^32 for the small type
  if (items <= (int64_t)1 << 31)
    paged_store_kernel<uint32_t><<<(unsigned)grid, 256, 0, stream>>>(p);
  else
    paged_store_kernel<int64_t><<<(unsigned)grid, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SDK_OK : SDK_ERR_CUDA;
}

}  // namespace sdk
