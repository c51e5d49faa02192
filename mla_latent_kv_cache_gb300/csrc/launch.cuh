// Internal launch interface shared by the C ABI layer and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace mla {

// Sets a kernel's attribute once per device (a driver call on every launch is a
// fifth of a small call); `done` is the kernel's own, a bit for each device.
inline cudaError_t attribute_once(std::atomic<uint64_t>& done, const void* kernel, cudaFuncAttribute attr, int value) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, attr, value);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Launch configuration that lets the grid start while the previous kernel
// in the stream drains (the kernel calls griddep_wait() before touching
// global memory that kernel may use).
inline cudaLaunchConfig_t pdl_config(dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                     cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Per-CTA status record (int32 words): 0 status bits, 1 first wait site,
// 2 its tile, 4 + role: (site << 24) | tile where that role gave up.
constexpr int kStatusRecWords = 16;

// Everything a decode launch needs; passed by value as a kernel parameter.
struct DecodeParams {
    const __nv_bfloat16* q_lat;
    const __nv_bfloat16* q_pe;
    const uint8_t* cache;
    int64_t num_slots;
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* seq_lens;
    void* out;
    float* lse;
    int* status;       // workspace header: status summary written by the merge step
    int* rec;          // [CTAs][kStatusRecWords] per-CTA status records
    float* part_o;     // [GY][SPG][64][lat_dim] fp32 partial outputs
    float* part_lse;   // [GY][SPG][64] fp32 partial LSEs
    float scale_log2;  // softmax scale * log2(e)
    int page_size;
    int run_rows;      // TMA box height: gcd(page_size, tile)
    int tile_shift;    // log2 of the tokens per tile: 7 (cluster kernel) or 6 (folded tiles)
    int B, Qt, Hq, HQ; // HQ = Hq * Qt rows per request (the largest Qt when cu_q is given)
    int out_f32;
    int SPG;           // partial slots per row group = workers + B
    int wseg;          // work-split cost of a request boundary, in tiles
    int test_hold;     // test hooks: 1 = withhold the first hand-off to the PV issuers,
                       // 2 = hold one PV issuer ~20 us after each of its first 32 tiles
    const int32_t* cu_q;  // [B + 1] prefix sums of query tokens per request, or null: Qt each
    int total_q;          // query tokens in q_lat, q_pe, out and lse; cu_q is clamped to [0, total_q]
    int lat_dim;       // latent width D: 512 (576-value rows), or 256 / 768 / 1792 (folded tiles, bf16)
    int rope_dim;      // rotary width P: 64
    int sms;           // of the device
    int64_t bt_cols;       // page-scaled rows: columns of the table
    const float* scales;   // and the pages' scales
};

cudaError_t launch_cache_write(const void* latent, int64_t latent_stride, const void* k_pe, int64_t k_pe_stride,
                               const int64_t* slot_mapping, int64_t num_tokens, void* cache, int64_t num_slots,
                               int kind, int* status, cudaStream_t stream);
// bf16 rows of another latent width D (2 (D + 64) bytes) (mla_cache_write_latent).
cudaError_t launch_cache_write_latent(const void* latent, int64_t latent_stride, const void* k_pe,
                                      int64_t k_pe_stride, const int64_t* slot_mapping, int64_t num_tokens,
                                      void* cache, int64_t num_slots, int lat_dim, int* status, cudaStream_t stream);
// Context gather of an fp8_ds_mla pool into bf16 rows (mla_gather_upconvert).
cudaError_t launch_gather_upconvert(const void* cache, int64_t num_slots, int page_size, const int32_t* block_table,
                                    int64_t bt_stride, const int32_t* cu_seq_lens, int B, int64_t num_rows, void* dst,
                                    int64_t dst_stride, cudaStream_t stream);
// Clusters (of 2 CTAs) the decode kernel variant runs with: the number that
// fit on the current device at once, or requested_ctas / 2 when given.
int decode_clusters(int NP, bool lsu, int kind, int requested_ctas);
// TMA descriptors of one decode call, unused when the load/convert warps
// read the pool. bf16 pools: lat = 64-dim latent chunks (128-B swizzle),
// rope = 32-dim rope halves (64-B swizzle). fp8 pools: lat = 256 code bytes
// of a row, aux = its 16 scale bytes, rope = 32-dim rope halves. q / qpe:
// 64-dim chunks of q_lat and 32-dim halves of q_pe, NP rows high.
struct DecodeMaps {
    CUtensorMap lat, aux, rope, q, qpe;
};

// Whether the folded-tile kernel has a variant for NP query rows, this latent
// width, cache kind and number of row groups.
bool fold_supported(int NP, int lat_dim, int kind, int GY);
// Whether that variant's workers are clusters of two CTAs (latent 1792).
bool fold_is_pair(int lat_dim);
// Workers of the folded-tile decode kernel (bf16 pools, page_size % 8 == 0)
// for GY row groups: the number that fit at once, or what requested_ctas CTAs
// make (a worker is a cluster of two for latent 1792, and for 65..128 query
// rows of the 576-wide row, whose two row groups share each tile).
int decode_fold_ctas(int NP, int lat_dim, int kind, int GY, int requested_ctas);
cudaError_t launch_decode_fold(const DecodeMaps& maps, const DecodeParams& p, int NP, int kind, int W, int GY,
                               cudaStream_t stream);
cudaError_t launch_decode(const DecodeMaps& maps, const DecodeParams& p, int NP, bool lsu, int kind, int G, int GY,
                          cudaStream_t stream);
// The merge of a decode's partial results over W workers (nrec status records).
cudaError_t launch_decode_merge(const DecodeParams& p, int W, int nrec, int GY, cudaStream_t stream);
// Rows with one scale for each page (mla_decode_fp8_page): maps.lat = 128 codes
// of a row (128-B swizzle), maps.rope = its 64 rotary codes (64-B swizzle), both
// gcd(page_size, 128) rows high; lsu: pages read row by row.
cudaError_t launch_decode_page8(const DecodeMaps& maps, const DecodeParams& p, int NP, bool lsu, int W, int GY,
                                cudaStream_t stream);
cudaError_t launch_merge_lse(const float* part_o, const float* part_lse, int S, int64_t N, void* out, int out_f32,
                             float* lse, cudaStream_t stream);

// Attention weights per cached token (mla_attn_weights).
struct WeightsParams {
    const __nv_bfloat16* q_lat;
    const __nv_bfloat16* q_pe;
    const float* lse;
    const uint8_t* cache;
    int64_t num_slots;
    int row_bytes;
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* seq_lens;
    float* weights;
    int64_t w_stride;
    int max_len;       // weights kept per request
    float decay;
    float scale_log2;  // softmax scale * log2(e)
    int page_size;
    int run_rows;      // TMA box height: gcd(page_size, 128)
    int B, Qt, Hq, HQ;
    int lat_dim;
    int np;            // query rows per group, padded (weights_plan)
    int groups;
    int slots;         // ring blocks
    int* status;
};
// rows: 64-dim blocks of a bf16 row or 128-code blocks of an fp8 one (128-B
// swizzle); fp8: rope = the 64 bf16 values at byte 528, scales = the 16 bytes
// at 512.
struct WeightsMaps {
    CUtensorMap rows, rope, scales;
};
bool weights_plan(int HQ, int lat_dim, int kind, WeightsParams& p, int* smem_bytes);
cudaError_t launch_attn_weights(const WeightsMaps& maps, const WeightsParams& p, int kind, bool lsu, int ctas,
                                int smem_bytes, cudaStream_t stream);

// Eviction by score (mla_cache_evict).
struct EvictParams {
    uint8_t* cache;
    int64_t num_slots;
    int row_bytes;
    int page_size;
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* seq_lens;
    const float* weights;
    const int32_t* positions;
    int64_t stride;    // of weights, positions and their new ones
    int max_len;
    const int32_t* budgets;
    int B;
    int n_sink, n_recent;
    int32_t* new_lens;
    float* new_weights;
    int32_t* new_positions;
    int32_t* moves;
    int64_t moves_stride;
    int* status;
};
constexpr int kMoveReqs = 1536;  // requests whose counts of moves a CTA of the move kernel holds at once
// Requests whose moves are counted at once: so many that 32 bits hold the sum.
// (A request moves at most min(K, T - K) <= max_len / 2 rows.)
constexpr int evict_requests_at_once(int max_len) {
    const uint32_t each = static_cast<uint32_t>(max_len) / 2;
    return each <= UINT32_MAX / kMoveReqs ? kMoveReqs : static_cast<int>(UINT32_MAX / each);
}
// most_ctas > 0: no more CTAs share a request's tokens (a test's; else as many as the device can run).
cudaError_t launch_evict(const EvictParams& p, int sms, int most_ctas, cudaStream_t stream);

// Attention over whole prompts (mla_prefill); strides in elements.
struct PrefillParams {
    const __nv_bfloat16* q;
    int64_t q_st, q_sh;
    const __nv_bfloat16* k_nope;
    int64_t k_st, k_sh;
    const __nv_bfloat16* k_pe;
    int64_t kp_st;
    const __nv_bfloat16* v;
    int64_t v_st, v_sh;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int B, total_q, total_k, Hq, Hkv;
    int pack;          // query heads that share a tile (prefill_pack)
    int tile_tokens;   // tokens of a tile: 128 / pack
    int causal;
    float scale_log2;  // softmax scale * log2(e)
    __nv_bfloat16* out;
    float* lse;
    int* status;
};
// 64-value blocks (128-B swizzle): q of tile_tokens tokens of pack heads, the
// others of one head: 128 tokens of keys, 64 of values.
struct PrefillMaps {
    CUtensorMap q, k_nope, k_pe, v;
};
int prefill_pack(int group);
int64_t prefill_pairs(int64_t total_q, int B, int max_q_len, int tile_tokens);
cudaError_t launch_prefill(const PrefillMaps& maps, const PrefillParams& p, int max_q_len, cudaStream_t stream);

// Rotary positions (mla_rope); strides in elements.
struct RopeParams {
    const void* x;
    int64_t x_t, x_h;
    void* out;
    int64_t o_t, o_h;
    const int32_t* positions;
    const int64_t* steps;
    int64_t T;
    int H, R;
    int interleaved;
    float mscale;
    int chunks, items_chunk;  // set by launch_rope: warps a token, 16-value items a warp
};
cudaError_t launch_rope(RopeParams p, int f32, int sms, cudaStream_t stream);

// New tokens into the paged cache (mla_cache_append); strides in elements.
struct AppendParams {
    const __nv_bfloat16* latent;
    int64_t lat_st;
    const __nv_bfloat16* k_pe;
    int64_t pe_st;
    const int32_t* cu;
    const int32_t* seq_lens;
    int B;
    int64_t total;
    const int32_t* block_table;
    int64_t bt_stride, bt_cols;
    int page_size;
    const int32_t* positions;   // or null: the place
    const int64_t* steps;       // or null: no rotation
    int interleaved;
    float mscale;
    const __nv_bfloat16* norm;  // or null
    float eps;
    uint8_t* cache;
    int64_t num_slots;
    float* scales;              // page rows
    __nv_bfloat16* rows;        // or null
    int64_t rows_st;
    int* status;
};
cudaError_t launch_append(const AppendParams& p, int kind, int lat_dim, int sms, cudaStream_t stream);

}  // namespace mla
