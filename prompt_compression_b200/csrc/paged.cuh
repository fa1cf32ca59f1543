// paged.cuh -- parameters of the paged-cache operators (pages.cu, tree.cu)
// and their host launchers.
//
// The cache: k_pages, v_pages [layers][n_pages][hkv][page_rows][head_dim];
// row t of sequence s is row t % page_rows of page
// page_table[s][t / page_rows], for every layer and KV head; seq_lens[s] rows
// are valid; page_refs[p] sequences hold page p (0: free).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace spk {

// ---------------------------------------------------------------- pages.cu
constexpr int kPagesMaxCall = 1024;   // sequences in one call

struct PagesShape {
  int layers, n_pages, hkv, page_rows;
  int row_vecs;            // 16-byte vectors of a row
  int n_seqs, max_pages;
};

struct PagesBook {         // the bookkeeping arrays
  int* refs;               // [n_pages]
  int* table;              // [n_seqs][max_pages]
  int* lens;               // [n_seqs]
};

size_t pages_ws_bytes(int n, int max_pages);

cudaError_t launch_pages_reserve(const PagesShape& s, const PagesBook& b, void* k_pages, void* v_pages,
                                 const int* seqs, const int* n_new, int n, int* result, void* ws,
                                 cudaStream_t stream);
cudaError_t launch_pages_fork(const PagesShape& s, const PagesBook& b, const int* src, const int* dst,
                              const int* n_rows, int n, int* result, void* ws, cudaStream_t stream);
cudaError_t launch_pages_free(const PagesShape& s, const PagesBook& b, const int* seqs, const int* keep_rows, int n,
                              cudaStream_t stream);
cudaError_t launch_pages_write(const PagesShape& s, const PagesBook& b, const void* k, const void* v, int n_src,
                               const int* idx, int n_idx, int units_per_idx, const int* counts, const int* seqs,
                               int n, void* k_pages, void* v_pages, const int* reserved, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesShape& s, const PagesBook& b, void* k_pages, void* v_pages,
                                 const int* src, const int* dst, int n, const int* idx, int n_idx,
                                 int units_per_idx, int* result, void* ws, cudaStream_t stream);
cudaError_t device_errors_pages(int* code, int* site, bool clear);

// ---------------------------------------------------- tree.cu, tree_umma.cu
constexpr int kTreeMaxBatch = 1024;
constexpr int kTreeMaxNodes = 1024;
constexpr int kTreeItemJobs = 4;   // what starting an item costs, in jobs

struct TreeParams {
  const void* q;           // [batch][layers][hq][T][d]
  const void* v_tree;      // [batch][layers][hkv][T][d] or null
  void* out;               // like q
  float* lse2;             // [batch][layers][hq][T] or null
  const int* table;        // [n_seqs][max_pages]
  const int* lens;         // [n_seqs]
  const int* seqs;         // [batch] or null (batch element b is sequence b)
  const int* n_live;       // [batch] or null (every node is live)
  const uint32_t* mask;    // [batch][T][words] or null (node i sees the nodes 0 .. i)
  int words;
  int batch, layers, hkv, T;
  int rows;                // query rows per unit = g * T, ordered [query head][node]
  int tile_rows;           // query rows of a row tile (wide kernel: 128)
  int row_tiles;           // row tiles per unit
  int items;               // items per unit
  int item_rows;           // rows of an item, in the partial results
  int has_tree;            // k_tree and v_tree are given
  int n_seqs, max_pages, n_pages, page_rows;
  int box_rows;            // rows of one page copy: divides page_rows and the key tile
  int node_rows;           // rows of one copy of nodes: min(T, key tile), a multiple of 8
  float c2;                // scale * log2(e)
  int ctas;                // CTAs of the main kernel
  int sms;
  bool join_inside;        // the main kernel joins the items that several shares hold
  float* part_o;           // [ctas * 2][d / 4][rows of an item][4] partial outputs
  float* part_ml;          // [ctas * 2][rows of an item][2] their row maxima and sums
  unsigned long long* arrived;   // [ctas] how many shares of a cut item are in, with the call's number
  unsigned long long call; // the call's number (48 bits)
};

struct TreePlan {
  bool wide;               // tree_umma.cu (row tiles of 128, two to an item) or tree.cu
  int keys;                // keys of a tile
  int tile_rows, row_tiles;
  int item_rows;           // query rows of an item
  int items;               // items per unit
  int ctas;
};
TreePlan tree_plan(int rows, int head_dim, int sms);
size_t tree_ws_bytes(const TreePlan& plan, int head_dim);

// maps: k_pages, v_pages [layers * n_pages * hkv][page_rows][d] in boxes of
// box_rows x 64; k_tree, v_tree [batch * layers * hkv][T][d] in boxes of
// node_rows x 64; q [batch * layers * hkv][rows][d] in boxes of 128 x 64 (wide only);
// k_pages, v_pages in boxes of 8 x 64
cudaError_t launch_tree_attention(bool fp16, int head_dim, const CUtensorMap (&maps)[7], const TreeParams& p,
                                  const TreePlan& plan, cudaStream_t stream);
cudaError_t launch_tree_umma(bool fp16, int head_dim, const CUtensorMap (&maps)[7], const TreeParams& p,
                             cudaStream_t stream);
// The main kernel alone, for bf16, head_dim 64 and units of up to 8 or 33 .. 128
// rows, with CTAs that lose work (spk_selftest_tree_give_up).
cudaError_t launch_tree_loses(const CUtensorMap (&maps)[7], const TreeParams& p, const TreePlan& plan, cudaStream_t stream);
cudaError_t launch_tree_umma_loses(const CUtensorMap (&maps)[7], const TreeParams& p, cudaStream_t stream);
cudaError_t launch_tree_mask(const int* parents, const int* n_live, int batch, int T, uint32_t* mask, int* depth,
                             cudaStream_t stream);
cudaError_t device_errors_tree(int* code, int* site, bool clear);
cudaError_t device_errors_tree_umma(int* code, int* site, bool clear);

}  // namespace spk
