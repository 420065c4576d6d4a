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
  int row0;       // first row of q
  int n;          // new tokens (0: idle or refused)
  int len;        // tokens in the store
  int lo;         // first token any row sees (by tiles: rounded down to one)
  int tile0;      // its first tile in the workspace
  int ntiles;
  int pair0;      // its first block of 256 packed rows (by atoms: first row pair)
  int npair;      // blocks per request and KV head (by atoms: pairs)
  int64_t work0;  // units of work before it: tiles of blocks (by atoms: tokens of pairs)
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
  ReqPlan* plan;         // [B + 1], the last one the totals
  // by tiles: running sums of the blocks' tiles (or parts), rebuilt key and value tiles
  // [tile][Hkv][tile image], partial sums [2 x CTA][256 rows][..]
  int64_t* units;
  char* cuts;            // what every share starts with
  __half* qt;            // scaled query tiles [block][Hkv][2][tile image]
  float* qscale;         // [block][Hkv][256 rows] score to log2 of its exponential
  __half* kt;
  __half* vt;
  float2* part_ml;
  float* part_o;
  // by atoms: <q, D_K> of row pairs [pair][n_pad], the rows' scales, scores
  // of (pair, token), and the weights per atom as operand images
  __half2* qd;
  float* row_scale;
  int4* pair_of;         // a pair's rows, and the first and last share of its tokens
  float2* score;
  char* wimg;
  int64_t n_tok, cap_pairs, cap_work;
  int B, Hq, Hkv, g, d, n, n_pad, n_pages, page_size, max_pages;
  int max_q, max_len, window, causal, cap_tiles;
  int ctas, sms, whole, parts, ksplits, row_tiles;
  float scale;
};

sdk_status launch_block_tables(const TableParams& p, cudaStream_t stream);
sdk_status launch_paged_store(const StoreParams& p, cudaStream_t stream);
// total_len as the caller's (0: B * max_len)
sdk_status launch_chunk_attn(ChunkParams p, int64_t total_len, char* workspace,
                             cudaStream_t stream);
// the other two forms (chunk_atoms.cu, chunk_direct.cu); by atoms: contexts of
// at most kAtomsMaxLen tokens, kAtomsMaxPairs row pairs over all KV heads and
// kAtomsMaxWork (row pair, token) units
constexpr int64_t kAtomsMaxLen = 1 << 24, kAtomsMaxPairs = 1 << 21, kAtomsMaxWork = (int64_t)1 << 35;
size_t atoms_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q,
                             int max_len, int64_t total_len);
sdk_status launch_chunk_atoms(ChunkParams p, int64_t total_len, char* workspace,
                              cudaStream_t stream);
bool direct_fits(int B, int64_t n_tok, int g, int max_q, int max_len);
size_t direct_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int max_q, int max_len,
                              int64_t total_len);
sdk_status launch_chunk_direct(ChunkParams p, int64_t total_len, char* workspace,
                               cudaStream_t stream);
// total bytes of the chunk attention's workspace
size_t chunk_workspace_bytes(int B, int64_t n_tok, int Hq, int Hkv, int d, int n, int max_q,
                             int max_len, int64_t total_len);
// most 128-token tiles the requests' contexts take
int64_t chunk_cap_tiles(int B, int max_len, int64_t total_len);

}  // namespace sdk
