// kernels.h -- internal interface between the C-ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sd {

constexpr int kSample = 2048;         // sampled positions per row for the candidate threshold
constexpr int kThresholdCluster = 8;  // CTAs (one cluster) that score one group's sample

struct TopkArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* K;
    const int32_t* page_table;
    const int32_t* lens;
    const int32_t* k;
    int32_t* idx;
    float* cand;        // workspace, B*Hq*n_cap floats: candidate scores, one sequential stream per
                        // score-pass warp; the candidates of one (page, head) are consecutive, in
                        // position order
    uint2* prec;        // workspace [B][Hq][mstride]: per (head, page) {where its candidates start in
                        // cand, 16-bit mask: bit i = position p*16 + i is a candidate}
    float* tau;         // workspace [B][Hq]: candidate threshold (scores >= tau are candidates;
                        // -inf: every position)
    const void** inputs;   // workspace [3]: q, K and page_table of the last score pass (the select
                           // step reads them from here when it has to recompute a row)
    int32_t* status;
    int B, Hq, Hkv, G, max_pages, num_pages, k_max;
    long n_cap;         // max_pages * page size: row stride of the score buffer
    int mstride;        // records per head row (max_pages rounded up to 8)
    int ccap;           // rows with N_b <= ccap take every position as a candidate
    int spp;            // pages per pipeline stage of the score pass
    int stages;         // pipeline depth of the score pass
    int cap;            // select: candidate entries that fit in shared memory
};

size_t score_pass_smem(const TopkArgs& a);
size_t threshold_smem(const TopkArgs& a);
cudaError_t launch_threshold(const TopkArgs& a, cudaStream_t stream);
size_t select_smem(const TopkArgs& a);
cudaError_t launch_score_pass(const TopkArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_select(const TopkArgs& a, cudaStream_t stream);

constexpr int kRange = 16384;           // dense decode: positions per counted range
constexpr int kMaxDecodeWarps = 1280;   // dense decode: persistent warps (one per CTA) at most
constexpr int kMaxSparseWarps = 4096;   // sparse decode: persistent warps (one per CTA) at most
constexpr int kRowSegs = 64;            // sparse decode: segment slots per (b, h) row
constexpr int kOrderMaxRows = 2048;     // sparse decode: rows up to which the offset order is used
constexpr int kRowBatch = 4;            // sparse decode: consecutive idx entries per rows_kernel thread and pass
constexpr uint32_t kSampledFlag = 0x40000000u;   // idx entry: a row drawn by the stochastic selection
constexpr int kPosMask = 0x3fffffff;             // the position bits of an idx entry

struct DecodeArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* K;
    const __nv_bfloat16* V;
    const int32_t* page_table;
    const int32_t* lens;
    const int32_t* idx;   // null for dense decode
    float* out;
    // workspace, sparse decode
    int* rlen;            // [B*Hq] entries before the first negative one
    int* arrive;          // [B*Hq] segments of the row finished so far (zeroed by rows_kernel)
    int* bsum;            // [nb] entries of the rows of each rows_kernel CTA
    float* rlw;           // [B*Hq] weighted mode: log2 of the weight of the row's drawn entries
    // workspace, dense decode and the sparse decode over GQA groups
    int* counts;          // [nrt] rows (positions) per range
    uint8_t* umask;       // sparse over groups: [B*Hkv][n_cap] heads of the group that selected each
                          // position (bit g: head kvh*G+g), 1 byte per position for G <= 8, else 2
    // workspace, both
    float2* ml;           // per (b, h, segment) running max (log2 units) and sum
    float* acc;           // per (b, h, segment) un-normalised output [128]
    int32_t* status;
    int B, Hq, Hkv, G, max_pages, num_pages, k_max;
    long n_cap;
    int nrp;              // dense: ranges per (b, kv head) group
    int nrt;              // dense: B * Hkv * nrp
    int tpr, rpc, nb;     // sparse: rows_kernel threads per row, rows per CTA, CTAs
    int min_epw;          // sparse: entries per warp at least (a row spans <= jmax warps)
    int jmax;             // segment slots per (b, h)
    int total_warps;      // persistent decode warps in the grid
    float scale_log2;     // log2(e) / sqrt(d)
    int weighted;         // sparse: idx entries with kSampledFlag are drawn rows of a stochastic
                          // selection, weighted by (N_b - plain entries) / drawn entries
    int order_rows;       // sparse: full rows are visited in offset order (heads of a group aligned)
    int union_tiles;      // group walk: whole 16-position tiles with head masks, instead of only the
                          // selected positions (the union covers nearly every position)
};

size_t decode_smem();
size_t sparse_decode_smem();
// CTAs (one warp each) of the decode kernel for (dense, G) that fit on one SM.
cudaError_t decode_occupancy(bool dense, int G, int* ctas_per_sm);
cudaError_t launch_sparse(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_sparse_union(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_dense(const DecodeArgs& a, cudaStream_t stream);

// Quest page-level indexer.
constexpr int kQuestMaxPages = 24 * 1024;   // pages per request the page select holds in shared memory

struct QuestArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* K;
    __nv_bfloat16* boxes;        // [num_pages][Hkv][2][128]: per-dimension minimum, then maximum
    const int32_t* page_table;
    const int32_t* lens;
    const int32_t* k;
    int32_t* idx;
    float* rel;                  // workspace [B][Hq][max_pages]: page relevance
    int32_t* status;
    int B, Hq, Hkv, G, max_pages, num_pages, k_max;
    long n_cap;
    int last_only;               // summarize: only each request's last page
};
cudaError_t launch_quest_summarize(const QuestArgs& a, cudaStream_t stream);
cudaError_t launch_quest_score(const QuestArgs& a, cudaStream_t stream);
cudaError_t launch_quest_select(const QuestArgs& a, cudaStream_t stream);
size_t quest_select_smem(const QuestArgs& a);

// Stochastic index selection: the draw from the rest of each row (stochastic.cu).
constexpr int kMaxSelectScratch = 64;   // ints of block-scan and selection state
struct SampleArgs {
    const int32_t* lens;
    const int32_t* k_det;
    const int32_t* k_samp;
    int32_t* idx;            // in: the exact top-k_det rows; out: those rows and the drawn ones
    int32_t* status;
    uint64_t seed;
    uint32_t step;
    int B, Hq, k_max;
    long n_cap;
    int words;               // 32-bit words of a bitmap over n_cap positions
    int cap;                 // candidate positions that fit in shared memory
};
size_t sample_smem(const SampleArgs& a);
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream);

struct AppendArgs {
    __nv_bfloat16* K;
    __nv_bfloat16* V;
    const int32_t* page_table;
    int32_t* lens;
    const __nv_bfloat16* k_new;
    const __nv_bfloat16* v_new;
    int32_t* k_sel;
    __nv_bfloat16* boxes;   // Quest boxes [num_pages][Hkv][2][128] kept up to date for the written page, or null
    int32_t* status;
    int B, Hkv, max_pages, num_pages, ratio;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);

// Ragged rows into a cache of any format and back (cache_io.cu).
struct CacheIoArgs {
    void* K;
    void* V;
    uint8_t* scales;          // 8-bit formats: [num_pages][Hkv][16][2][4], else null
    const int32_t* page_table;
    const int32_t* lens;
    const int32_t* first;     // read: first position of each request
    const int32_t* row_start; // [B + 1]
    const __nv_bfloat16* k_in;
    const __nv_bfloat16* v_in;
    __nv_bfloat16* k_out;     // read: either may be null
    __nv_bfloat16* v_out;
    __nv_bfloat16* boxes;     // write: Quest boxes of the written pages, or null
    int32_t* status;
    int B, Hkv, max_pages, num_pages, total_rows, sms;
    int parts;                // units that a run of rows in one page is taken in
    long n_cap;
};
cudaError_t launch_cache_write(const CacheIoArgs& a, int format, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheIoArgs& a, int format, cudaStream_t stream);

// Attention of a chunk of new positions over a cache of any format (chunk_attention.cu).
struct ChunkArgs {
    const __nv_bfloat16* q;   // [total_rows][Hq][128]
    const void* K;
    const void* V;
    const uint8_t* scales;
    const int32_t* page_table;
    const int32_t* lens;
    const int32_t* row_start;
    __nv_bfloat16* out;       // [total_rows][Hq][128]
    int32_t* status;
    // workspace: the parts of items that a CTA's border cuts, two slots of 256 rows per CTA
    float* part;              // un-normalised outputs
    float2* ml;               // maximum (log2 units) and sum of each row
    void* tail;               // per CTA: the item that goes on in later CTAs
    float* few_part;          // the same for cache_decode.cu, two slots of eight rows per share
    float2* few_ml;
    void* few_tail;
    int32_t* tiles;           // whether a request of this call is chunk_attention.cu's, where both take part
    int B, Hq, Hkv, G, max_pages, num_pages, total_rows, sms;
    int tpt;                  // tokens to a tile of 128 rows: 128 / G
    int few;                  // requests of at most so many new rows are cache_decode.cu's, the others chunk_attention.cu's
    long n_cap;
    float scale_log2;         // log2(e) / sqrt(d)
};
constexpr int kChunkCtas = 160;   // persistent CTAs at most
struct ChunkLayout {
    size_t part, ml, tail, few_part, few_ml, few_tail, tiles, total;
};
ChunkLayout chunk_layout();
cudaError_t launch_chunk_attention(const ChunkArgs& a, int format, cudaStream_t stream);
// The same for few rows per KV head over an 8-bit cache (cache_decode.cu).
constexpr int kDecodeShares = 2048;   // warps of one wave at most
cudaError_t launch_cache_decode(const ChunkArgs& a, int format, cudaStream_t stream);
cudaError_t launch_merge_decode(const ChunkArgs& a, cudaStream_t stream);

// Sparse decode over an 8-bit cache (cache_sparse.cu).
struct CacheSparseArgs {
    const __nv_bfloat16* q;
    const void* K;
    const void* V;
    const uint8_t* scales;
    const int32_t* page_table;
    const int32_t* lens;
    const int32_t* idx;
    float* out;
    // workspace: parts of rows that a share's border cuts, two slots per warp
    float* part;              // un-normalised outputs [128]
    float2* ml;               // maximum (log2 units) and sum
    int32_t* status;
    int B, Hq, Hkv, G, max_pages, num_pages, k_max, sms;
    int shares;               // warps that the slots of idx are cut over
    long n_cap;
    float scale_log2;
};
constexpr int kCacheSparseWarps = 4096;   // warps of one wave at most
cudaError_t launch_cache_sparse(const CacheSparseArgs& a, int format, cudaStream_t stream);

}  // namespace sd
