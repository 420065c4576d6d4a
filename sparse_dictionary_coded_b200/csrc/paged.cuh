// Parameter blocks and launchers of the paged code store's kernels.
#pragma once

#include "sdk_internal.cuh"

namespace sdk {

struct TableParams {
  const int32_t* lens;
  const int32_t* n_new;
  const int32_t* free_pages;
  const int32_t* n_free;
  int32_t* table;
  int64_t* slot_map;
  int32_t* cu_new;
  int32_t* new_lens;
  int32_t* n_free_out;
  WsHeader* hdr;
  int64_t max_new;
  int B, n_stack, n_pages, page_size, max_pages;
};

struct StoreParams {
  const uint32_t* codes_k;
  const uint32_t* codes_v;
  const int64_t* slot_map;
  uint32_t* pages;
  WsHeader* hdr;
  int64_t n_tok;
  int Hkv, n_pages, page_size;
};

// One request of a chunk call, as every kernel of the call sees it.
struct ReqPlan {
  int row0;     // first row of q
  int n;        // new tokens (0: idle or refused)
  int len;      // tokens in the store
  int lo;       // first token any row sees, rounded down to a tile
  int tile0;    // its first tile in the workspace
  int ntiles;
  int pad[2];
};

struct ChunkParams {
  const uint16_t* q;
  const uint16_t* dk;
  const uint16_t* dv;
  const uint32_t* pages;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu_q;
  uint16_t* out;
  float* lse;
  WsHeader* hdr;
  ReqPlan* plan;
  __half* kt;            // rebuilt key tiles [tile][Hkv][tile image]
  __half* vt;
  float2* part_ml;       // partial sums of the splits [split][row][..]
  float* part_o;
  int64_t n_tok;
  int B, Hq, Hkv, g, d, n, n_pages, page_size, max_pages;
  int max_q, max_len, window, causal, cap_tiles, mblocks, splits;
  float scale;
};

sdk_status launch_block_tables(const TableParams& p, cudaStream_t stream);
sdk_status launch_paged_store(const StoreParams& p, cudaStream_t stream);
sdk_status launch_chunk_attn(ChunkParams p, char* workspace, cudaStream_t stream);
// total bytes of the chunk attention's workspace
size_t chunk_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q,
                             int max_len, int64_t total_len);
// most 128-token tiles the requests' contexts take
int64_t chunk_cap_tiles(int B, int max_len, int64_t total_len);

}  // namespace sdk
