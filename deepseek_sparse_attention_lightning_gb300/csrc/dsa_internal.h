// dsa_internal.h -- declarations shared by the translation units of libdsa.so
// (launchers and device-error accessors).  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

struct dsa_decode_desc;

namespace dsa {

constexpr int kIndexHeads = 64;
constexpr int kIndexDim = 128;
constexpr int kLatentDim = 576;
constexpr int kVDim = 512;
constexpr int kPage = 64;
constexpr int kHistBins = 2048;     // top 11 bits of the order-preserving score key
constexpr int kHistShift = 21;
constexpr int kTopkChunk = 8192;    // logits per CTA in the top-k passes
constexpr int kTopkClusterCtas = 16;  // CTAs (chunks) per query row in the select pass
// Rows of up to 16 chunks of 4 x 8192 scores.
constexpr int64_t kTopkMaxLd = int64_t(kTopkClusterCtas) * kTopkChunk * 4;

struct IndexerLaunch {
  const uint8_t* q_fp8;
  const float* q_scale;
  const float* w;
  const uint8_t* k_fp8;
  const float* k_scale;
  const int32_t* seqlens;
  const int32_t* page_table;
  float* logits;
  int64_t ld;
  uint32_t* hist;       // [T][kHistBins] or nullptr
  int batch, nq, max_pages, num_pages, topk;
  int skip_short;       // skip requests whose queries all see <= topk tokens
  int pdl;              // 1: launched as a programmatic dependent of the workspace clear
  int wait_tail;        // 1: that kernel also writes new tokens' keys: each request's last
                        //    two tiles are read only after it completed
  long long wait_cycles;   // bound of the pipeline waits (set by launch_indexer)
};

struct TopkLaunch {
  const int32_t* seqlens;
  const float* logits;
  int64_t ld;
  int32_t* out;         // [T][k]
  uint32_t* hist;       // [T][kHistBins], zeroed (or filled by the indexer)
  uint2* cand;          // [T][ld]: chunk c's candidates at the chunk's first position
  int batch, nq, k;
  int hist_ready;       // 1: hist already holds the row histograms
  int pdl;              // 1: launched as a programmatic dependent of the indexer
};

struct CacheWriteLaunch {
  const uint16_t* new_latent;    // [T][576] bf16: the new tokens' latent rows
  const uint16_t* new_index_k;   // [T][128] bf16: the new tokens' indexer keys
  uint16_t* kv;                  // [num_pages * 64][576] bf16 latent cache
  uint8_t* k_fp8;                // [num_pages * 64][128] E4M3 indexer-key cache
  float* k_scale;                // [num_pages * 64] its per-token scales
  const int32_t* seqlens;
  const int32_t* page_table;
  int batch, nq, max_pages, num_pages;
  uint4* clear;                  // zero-filled by CTAs of their own, or nullptr
  long long clear_n16;           // its 16-byte words
};

struct MlaLaunch {
  const uint16_t* q;
  const uint16_t* kv;
  const uint8_t* kv8;   // non-null: the latent cache in FP8 rows of 656 bytes (kv unused)
  const int32_t* topk_idx;
  const int32_t* seqlens;
  const int32_t* page_table;
  float* mid_o;
  float* mid_lse;
  int batch, nq, heads, k, max_pages, num_pages, num_splits;
  float sm_scale;
  int pdl;              // 1: launched as a programmatic dependent of the top-k
  int sel_ready;        // 1: topk_idx was complete before the kernel this one depends on
                        //    started (read without waiting); with pdl the grid then
                        //    completes only after that kernel
};

struct RmsNormLaunch {
  const uint16_t* x;             // [rows] rows of dim bf16, ld_x apart
  const uint16_t* residual;      // [rows][dim] bf16 or nullptr
  const uint16_t* weight;        // [dim] bf16
  uint16_t* residual_out;        // [rows][dim] bf16 or nullptr
  uint16_t* y;                   // [rows][dim] bf16 or nullptr
  uint8_t* y8;                   // [rows][dim] E4M3 or nullptr
  float* y_scale;                // [rows][tiles] (with y8)
  long long rows, ld_x;
  int dim;
  int group;                     // 128: a scale for each 128 columns; 0: one a row
  float eps;
};

struct MlaDecodeLaunch {
  const uint16_t* q;             // [T][H][576] bf16
  const uint16_t* kv;            // [num_pages * 64][576] bf16
  const uint8_t* kv8;            // non-null: the latent cache in FP8 rows of 656 bytes (kv unused)
  const int32_t* seqlens;
  const int32_t* page_table;
  uint16_t* out;                 // [T][H][512] bf16
  float* lse;                    // [T][H] or nullptr
  float* part_o;                 // set by launch_mla_decode: partial outputs and
  float* part_lse;               //   their log-sum-exps, in the workspace, and for
  int2* joins;                   //   each group the request joined from it on
  int batch, nq, heads, max_pages, num_pages;
  int row_tiles, groups, min_tiles;   // set by launch_mla_decode
  float sm_scale;
};

struct MlaPrefillLaunch {
  const uint16_t* q;             // [total_q][H][192] bf16
  const uint16_t* kv;            // [total_k][H][256] bf16: key 128, value 128
  const uint16_t* k_rope;        // [total_k] rows of 64 bf16, ld_rope apart
  const int32_t* cu_q;           // [batch + 1]
  const int32_t* cu_k;
  uint16_t* out;                 // [total_q][H][128] bf16
  float* lse;                    // [total_q][H] or nullptr
  long long ld_rope;
  int batch, heads, total_q, total_k, max_q, causal;
  int out_wide;                  // set by launch_mla_prefill: out is 32-byte aligned
  int parts;                     //   CTAs (a cluster) that share an item's keys
  int slots, head_group;         //   query blocks of all requests; heads that run together
  float sm_scale;
};

struct PagesLaunch {
  const int32_t* change;         // [batch] tokens added; < 0: the request has ended
  const int32_t* seqlens;        // [batch]
  int32_t* seqlens_out;          // [batch], may be seqlens
  int32_t* page_table;           // [batch][max_pages]
  int32_t* free_pages;           // [num_pages], a stack
  const int32_t* free_count;     // pages on it
  int32_t* free_count_out;       // may be free_count
  int32_t* cu_new;               // [batch + 1]
  int32_t* slots;                // [max_tokens]
  int batch, max_pages, num_pages, max_tokens;
};

struct KvWriteLaunch {
  const uint16_t* k;             // [tokens] rows of kv_heads * dim bf16, ld_k apart
  const uint16_t* v;
  const int32_t* slots;          // [tokens] cache rows, -1: none
  void* k_cache;                 // [num_pages][kv_heads][64][dim] bf16, or E4M3 with scales
  void* v_cache;
  float* k_scale;                // [num_pages][kv_heads][64], or nullptr (bf16)
  float* v_scale;
  long long ld_k, ld_v;
  int tokens, kv_heads, dim, num_pages;
};

struct GqaPrefillLaunch {
  const uint16_t* q;             // [total_q] rows of heads * dim bf16, ld_q apart
  const uint16_t* k;             // [total_k] rows of kv_heads * dim bf16, ld_k apart
  const uint16_t* v;
  const int32_t* cu_q;           // [batch + 1]
  const int32_t* cu_k;
  uint16_t* out;                 // [total_q][heads][dim] bf16
  float* lse;                    // [total_q][heads] or nullptr
  long long ld_q, ld_k, ld_v;
  int batch, heads, kv_heads, dim, total_q, total_k, max_q, causal;
  int group, tile_q;             // set by launch_gqa_prefill: query heads a key head, queries of a tile
  int out_wide;                  //   out is 32-byte aligned
  int parts;                     //   CTAs (a cluster) that share an item's keys
  int first_item;                //   of the launch
  int slots, head_group;         //   query blocks of all requests; key heads that run together
  float sm_scale;
};

struct GqaDecodeLaunch {
  const uint16_t* q;             // [T][heads][dim] bf16
  const void* k;                 // [num_pages][kv_heads][64][dim] bf16, or E4M3 with scales
  const void* v;
  const float* k_scale;          // [num_pages][kv_heads][64], or nullptr (bf16)
  const float* v_scale;
  const int32_t* seqlens;
  const int32_t* page_table;
  uint16_t* out;                 // [T][heads][dim] bf16
  float* lse;                    // [T][heads] or nullptr
  float* part_o;                 // set by launch_gqa_decode: partial outputs and
  float* part_lse;               //   their log-sum-exps, in the workspace, and for
  int4* joins;                   //   each CTA what is joined from it on
  int batch, nq, heads, kv_heads, dim, max_pages, num_pages;
  int row_tiles, tile_q, tile_rows, ctas, min_tiles;   // set by launch_gqa_decode
  float sm_scale;
};

cudaError_t launch_indexer(const IndexerLaunch& a, cudaStream_t s);
// Bound, in SM cycles, of the indexer's pipeline waits on later launches
// (<= 0: the default kWaitCycles).
void set_indexer_wait_cycles(long long cycles);
cudaError_t launch_topk(const TopkLaunch& a, cudaStream_t s);
cudaError_t launch_sparse_mla(const MlaLaunch& a, cudaStream_t s);
cudaError_t launch_cache_write(const CacheWriteLaunch& a, cudaStream_t s);
cudaError_t launch_latent_fp8(const uint16_t* kv, long long rows, uint8_t* kv8, cudaStream_t s);
cudaError_t launch_rmsnorm(const RmsNormLaunch& a, cudaStream_t s);
// Dense latent attention: its plan (row tiles of a request, groups of CTA
// pairs, workspace bytes; no kernel) and its launch.
void mla_decode_plan(int nq, int heads, int* row_tiles, int* groups, size_t* ws_bytes);
cudaError_t launch_mla_decode(MlaDecodeLaunch a, void* ws, cudaStream_t s);
// Prompt attention: blocks of its grid before keys are shared (at most INT_MAX;
// no kernel), and its launch.
long long mla_prefill_items(const MlaPrefillLaunch& a);
cudaError_t launch_mla_prefill(MlaPrefillLaunch a, cudaStream_t s);
cudaError_t launch_pages(const PagesLaunch& a, cudaStream_t s);
cudaError_t launch_kv_write(const KvWriteLaunch& a, cudaStream_t s);
// Prompt attention with grouped heads: blocks of its grid before keys are shared
// (no kernel), and its launch.
long long gqa_prefill_items(const GqaPrefillLaunch& a);
cudaError_t launch_gqa_prefill(GqaPrefillLaunch a, cudaStream_t s);
// Paged attention with grouped heads: its workspace (no kernel), and its launch.
size_t gqa_decode_workspace(int dim);
cudaError_t launch_gqa_decode(GqaDecodeLaunch a, void* ws, cudaStream_t s);
cudaError_t launch_merge(int rows, int splits, const float* mid_o, const float* mid_lse,
                         float* out, float* out_lse, cudaStream_t s, bool pdl = false);

// Launches `kern` on `s`; with `pdl` as a programmatic dependent of the
// previous kernel of the stream (the kernel then calls grid_dep_wait before it
// reads anything that kernel wrote).
// `cluster_x` > 1 groups consecutive CTAs along x into clusters of that size.
template <typename... Exp, typename... Act>
cudaError_t launch_kernel(void (*kern)(Exp...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t s, bool pdl, int cluster_x, Act&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster_x);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Act&&>(args)...);
}

// Each translation unit keeps its own device error word (0 or a dsa_status code);
// these give its address on the current device, or nullptr.
int* error_word_indexer();
int* error_word_topk();
int* error_word_mla();
int* error_word_merge();
int* error_word_cache();
int* error_word_mla_dense();
int* error_word_mla_prefill();
int* error_word_pages();
int* error_word_kv_write();
int* error_word_gqa_prefill();
int* error_word_gqa_decode();

// Host helpers (dsa_api.cu).
// The checks every entry point applies to a decode descriptor: a dsa_status.
int check_decode_desc(const ::dsa_decode_desc* d);
bool encode_tmap_2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base,
                    uint64_t inner, uint64_t outer, uint64_t row_bytes, uint32_t box_inner,
                    uint32_t box_outer, CUtensorMapSwizzle swizzle);
// Rank-r map (r <= 5): dims[0] is contiguous, byte_strides[i] is the stride
// of dimension i + 1; no fill for out-of-range loads, clipped stores.
bool encode_tmap_nd(CUtensorMap* map, CUtensorMapDataType dtype, const void* base, int rank,
                    const uint64_t* dims, const uint64_t* byte_strides, const uint32_t* box,
                    CUtensorMapSwizzle swizzle);
int device_sm_count();

}  // namespace dsa

// Defines the per-TU device error word and what gives its address.
#define DSA_DEFINE_ERROR_WORD(NAME)                                                    \
  namespace dsa {                                                                      \
  static __device__ int g_error_word = 0;                                              \
  __device__ __forceinline__ void raise_error(int code) {                              \
    atomicCAS(&g_error_word, 0, code);                                                 \
  }                                                                                    \
  int* error_word_##NAME() {                                                           \
    void* at = nullptr;                                                                \
    return cudaGetSymbolAddress(&at, g_error_word) == cudaSuccess ? static_cast<int*>(at) : nullptr; \
  }                                                                                    \
  }
