// qmm_launch.h -- internal host launchers (called by api.hip after validation).
// Arguments are already checked: sizes in range, K a multiple of the block,
// pointers non-null and 16-byte aligned.  Each returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace qmm {

// Opts kernel `func` into `bytes` of dynamic LDS (past the default 64 KiB)
// once per device: `done` holds one bit per device id below 64 (higher ids
// set the attribute on every call).  The attribute call is idempotent and the
// mask atomic, so concurrent first calls from several threads are safe.
inline hipError_t ensure_lds_bytes(const void *func, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return hipSuccess;
    e = hipFuncSetAttribute(func, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess && bit != 0) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

hipError_t launch_quantize_q8_0(const float *x, uint8_t *y, int64_t M, int64_t K, hipStream_t s);
hipError_t launch_quantize_q8_K(const float *x, uint8_t *y, int64_t M, int64_t K, hipStream_t s);
hipError_t launch_encode_q4_0(const float *w, uint8_t *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_encode_q4_K(const float *w, uint8_t *out, int64_t N, int64_t K, hipStream_t s);

int64_t repacked_bytes_q4_0(int64_t N, int64_t K);
int64_t repacked_bytes_q6_K(int64_t N, int64_t K);
hipError_t launch_repack_q4_0(const uint8_t *in, uint8_t *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_repack_q4_K(const uint8_t *in, uint8_t *out, int64_t N, int64_t K, hipStream_t s);

// GEMV family: M <= 8.  `repacked` selects the weight layout.
hipError_t launch_gemv_q4_0(const uint8_t *w, bool repacked, const uint8_t *y, float *out,
                            int64_t M, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemv_q4_K(const uint8_t *w, bool repacked, const uint8_t *y, float *out,
                            int64_t M, int64_t N, int64_t K, hipStream_t s);
// Fused M = 1 quantize + GEMV: x is one fp32 row of K values; yq receives its
// Q8_K bytes.  Valid for K <= gemv1_fused_max_k().
int64_t gemv1_fused_max_k();
hipError_t launch_gemv1_fused_q4_K(const uint8_t *w, bool repacked, const float *x, uint8_t *yq,
                                   float *out, int64_t N, int64_t K, hipStream_t s);
// int32 per-(sub-)block sums with the GEMV decode path (verification aid).
hipError_t launch_block_sums_q4_0(const uint8_t *w, bool repacked, const uint8_t *y, int32_t *P,
                                  int64_t M, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_block_sums_q4_K(const uint8_t *w, bool repacked, const uint8_t *y, int32_t *P,
                                  int64_t M, int64_t N, int64_t K, hipStream_t s);

// Small-batch MFMA family: M <= skinny_max_m(), weight and activation
// matrices below 4 GiB (32-bit buffer offsets).
int64_t skinny_max_m();
hipError_t launch_skinny_q4_K(const uint8_t *w, bool repacked, const uint8_t *y, float *out,
                              int64_t M, int64_t N, int64_t K, hipStream_t s);
// The same on 16 x 16 MFMA tiles (workgroups of 16 rows and 16 or 32
// columns): M <= skinny16_max_m(), matrices below 4 GiB.
int64_t skinny16_max_m();
// compute units of the current device (queried once per device)
int cu_count();
// Q4_K small batch, repacked layout, 1 <= M <= 8 (skinny16r.hip): producer
// wavefront streaming through an LDS ring, four consumer wavefronts.
hipError_t launch_skinny16r_q4_K(const uint8_t *w, const uint8_t *y, float *out, int64_t M, int64_t N,
                                 int64_t K, hipStream_t s);
// Q4_K small batch, repacked layout, 1 <= M <= 32 (skinny32r.hip): two or three
// producer wavefronts streaming through an LDS ring, four consumer wavefronts.
hipError_t launch_skinny32r_q4_K(const uint8_t *w, const uint8_t *y, float *out, int64_t M, int64_t N,
                                 int64_t K, hipStream_t s);
hipError_t launch_skinny16_q4_K(const uint8_t *w, bool repacked, const uint8_t *y, float *out,
                                int64_t M, int64_t N, int64_t K, hipStream_t s);
// Q4_0, M = 1, small matrices (gemv_fused_q4_0_ok): quantize + GEMV in one launch
bool gemv_fused_q4_0_ok(int64_t N, int64_t K);
hipError_t launch_gemv_fused_q4_0(const uint8_t *w, bool repacked, const float *x, uint8_t *yq, float *out,
                                  int64_t N, int64_t K, hipStream_t s);
// Q6_K, M = 1, K <= 8192, N <= 32 * CUs (gemv_fused_q6_K_ok): quantize + GEMV in one launch
bool gemv_fused_q6_K_ok(int64_t N, int64_t K);
hipError_t launch_gemv_fused_q6_K(const uint8_t *w, bool repacked, const float *x, uint8_t *yq, float *out,
                                  int64_t N, int64_t K, hipStream_t s);
// Q2_K, M = 1, K <= 16384, N <= 32 * CUs (gemv_fused_q2_K_ok): quantize + GEMV in one launch
bool gemv_fused_q2_K_ok(int64_t N, int64_t K);
hipError_t launch_gemv_fused_q2_K(const uint8_t *w, bool repacked, const float *x, uint8_t *yq, float *out,
                                  int64_t N, int64_t K, hipStream_t s);
// Q4_0 GEMV with the M activation rows staged in LDS: K % 64 == 0 and
// M * K * 5/4 bytes <= 60 KiB (other shapes read the rows per lane).
bool gemv_q4_0s_fits(int64_t M, int64_t K);
// Q4_0 small batch: repacked layout, K % 256 == 0, M <= skinny_q4_0_max_m(),
// matrices below 4 GiB; w_bytes is the repacked matrix size.
int64_t skinny_q4_0_max_m();
hipError_t launch_skinny_q4_0(const uint8_t *w, int64_t w_bytes, const uint8_t *y, float *out, int64_t M,
                              int64_t N, int64_t K, hipStream_t s);

// Q6_K (encoder, load-time repack, GEMV for any M with K <= q6_K_max_k(),
// int32 group sums P[m][n][K/16] of the same decode path).
int64_t q6_K_max_k();
hipError_t launch_encode_q6_K(const float *w, uint8_t *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_repack_q6_K(const uint8_t *in, uint8_t *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemv_q6_K(const uint8_t *w, bool repacked, const uint8_t *y, float *out,
                            int64_t M, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_group_sums_q6_K(const uint8_t *w, bool repacked, const uint8_t *y, int32_t *P,
                                  int64_t M, int64_t N, int64_t K, hipStream_t s);

// Q2_K (encoder, load-time repack, GEMV for any M with K <= q2_K_max_k(),
// int32 group sums P[m][n][K/16] of the same decode path).
int64_t repacked_bytes_q2_K(int64_t N, int64_t K);
int64_t q2_K_max_k();
hipError_t launch_encode_q2_K(const float *w, uint8_t *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_repack_q2_K(const uint8_t *in, uint8_t *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemv_q2_K(const uint8_t *w, bool repacked, const uint8_t *y, float *out,
                            int64_t M, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_group_sums_q2_K(const uint8_t *w, bool repacked, const uint8_t *y, int32_t *P,
                                  int64_t M, int64_t N, int64_t K, hipStream_t s);
// both group-sum paths stage one activation row in LDS
inline int64_t q8k_group_max_k() { return q6_K_max_k() < q2_K_max_k() ? q6_K_max_k() : q2_K_max_k(); }

// MFMA GEMM family (any M >= 1; weight and activation matrices below 4 GiB:
// 32-bit buffer offsets).  The Q6_K and Q2_K GEMMs take the repacked layout
// of w_bytes bytes.
hipError_t launch_gemm_q4_K(const uint8_t *w, bool repacked, const uint8_t *y, float *out,
                            int64_t M, int64_t N, int64_t K, hipStream_t s);
// Q6_K small batch: repacked layout, M <= skinny_q6_K_max_m(), matrices below
// 4 GiB; w_bytes is the repacked matrix size.
int64_t skinny_q6_K_max_m();
hipError_t launch_skinny_q6_K(const uint8_t *w, int64_t w_bytes, const uint8_t *y, float *out, int64_t M,
                              int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemm_q6_K(const uint8_t *w, int64_t w_bytes, const uint8_t *y, float *out,
                            int64_t M, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemm_q2_K(const uint8_t *w, int64_t w_bytes, const uint8_t *y, float *out,
                            int64_t M, int64_t N, int64_t K, hipStream_t s);
// Q2_K small batch: repacked layout, M <= skinny_q2_K_max_m(), matrices below
// 4 GiB; w_bytes is the repacked matrix size.
int64_t skinny_q2_K_max_m();
hipError_t launch_skinny_q2_K(const uint8_t *w, int64_t w_bytes, const uint8_t *y, float *out, int64_t M,
                              int64_t N, int64_t K, hipStream_t s);
// Q4_0 x Q8_0, repacked layout, K a multiple of 256.
hipError_t launch_gemm_q4_0(const uint8_t *w, int64_t w_bytes, const uint8_t *y, float *out,
                            int64_t M, int64_t N, int64_t K, hipStream_t s);

constexpr int kGemvMaxM = 8;

// ---- mul_mat_id (Q4_K).  The expert grouping lives in a caller workspace of
// int32 words: start[E+1] (first sorted slot of each expert), tile_e and
// tile_r0 [max_tiles] (expert and first sorted slot of each GEMM row tile),
// ntiles[1], sorted[P] (pair index per sorted slot), each section aligned to
// 16 bytes.  Each expert adds at most one partial tile, so max_tiles =
// ceil(P / bm) + E.
struct MoeGroupLayout {
    int64_t start, tile_e, tile_r0, ntiles, sorted, max_tiles, words;
};
inline MoeGroupLayout moe_group_layout(int64_t P, int64_t E, int64_t bm) {
    auto up4 = [](int64_t v) { return (v + 3) / 4 * 4; };
    MoeGroupLayout L;
    L.max_tiles = (P + bm - 1) / bm + E;
    L.start = 0;
    L.tile_e = L.start + up4(E + 1);
    L.tile_r0 = L.tile_e + up4(L.max_tiles);
    L.ntiles = L.tile_r0 + up4(L.max_tiles);
    L.sorted = L.ntiles + 4;
    L.words = L.sorted + up4(P);
    return L;
}
constexpr int kMoeMaxExperts = 4096;
int gemm_tile_rows();  // BM of the Q4_K GEMM
int64_t gemv1_max_k();
// The library's own grouping area for callers that cannot allocate: device
// address of a static array of kNoAllocScratchBytes on the device of `stream`
// (the current device for the null stream), looked up once per device.
constexpr size_t kNoAllocScratchBytes = size_t(2) << 20;
hipError_t noalloc_scratch(hipStream_t stream, int32_t **ptr);
// Build the grouping for pairs p < P with expert ids[p] (ids outside [0, E)
// are left out, and their output rows are filled with NaN).
hipError_t launch_moe_group_ids(const int32_t *ids, int64_t P, int64_t E, int32_t *ws, float *out,
                                int64_t N, hipStream_t s);
// M = 1 GEMV per (token, slot) pair; w_stride = bytes per expert matrix.
hipError_t launch_gemv_id_q4_K(const uint8_t *w, bool repacked, int64_t w_stride, const uint8_t *y,
                               int y_per_slot, const int32_t *ids, int64_t P, int64_t U, int64_t E,
                               float *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemv_id_q6_K(const uint8_t *w, bool repacked, int64_t w_stride, const uint8_t *y,
                               int y_per_slot, const int32_t *ids, int64_t P, int64_t U, int64_t E,
                               float *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemv_id_q2_K(const uint8_t *w, bool repacked, int64_t w_stride, const uint8_t *y,
                               int y_per_slot, const int32_t *ids, int64_t P, int64_t U, int64_t E,
                               float *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemv_id_q4_0(const uint8_t *w, bool repacked, int64_t w_stride, const uint8_t *y,
                               int y_per_slot, const int32_t *ids, int64_t P, int64_t U, int64_t E,
                               float *out, int64_t N, int64_t K, hipStream_t s);
// The GEMMs over the grouped tiles (after launch_moe_group_ids on ws); the
// Q6_K, Q2_K and Q4_0 ones take the repacked layout, w_bytes = one expert.
hipError_t launch_gemm_id_q6_K(const uint8_t *w, int64_t w_bytes, const uint8_t *y, int64_t y_rows,
                               int y_per_slot, int64_t U, const int32_t *group_ws, int64_t E, int64_t P,
                               float *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemm_id_q2_K(const uint8_t *w, int64_t w_bytes, const uint8_t *y, int64_t y_rows,
                               int y_per_slot, int64_t U, const int32_t *group_ws, int64_t E, int64_t P,
                               float *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemm_id_q4_0(const uint8_t *w, int64_t w_bytes, const uint8_t *y, int64_t y_rows,
                               int y_per_slot, int64_t U, const int32_t *group_ws, int64_t E, int64_t P,
                               float *out, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_gemm_id_q4_K(const uint8_t *w, bool repacked, int64_t w_stride, const uint8_t *y,
                               int64_t y_rows, int y_per_slot, int64_t U, const int32_t *group_ws,
                               int64_t E, int64_t P, float *out, int64_t N, int64_t K, hipStream_t s);

// ---- rows of a packed table by id, decoded and scaled (embed.hip); fmt is a qmm_weight_type
hipError_t launch_embed_rows(int fmt, const uint8_t *w, bool repacked, const int32_t *ids, int64_t T, float scale,
                             float *out, int64_t N, int64_t K, hipStream_t s);
bool embed_rows_long(int64_t T, int64_t K);  // the output goes past the caches

// ---- low-rank adapters per row (lora.hip); type is a qmm_float_type (of A and B).
// Workspace: fp32 partial sums of v[m][r], one set per split of K.
struct LoraArgs {
    const void *A, *B;      // [E][R][K], [E][N][R]
    const float *scales;    // [E] or null (1)
    const int32_t *ranks;   // [E] or null (R)
    const float *x;         // [M][K]
    const int32_t *ids;     // [M]
    const float *base;      // row stride ld_base; may be out
    float *out;             // row stride ld_out
    float *ws;
    int64_t M, N, K, R, E, ld_base, ld_out;
};
int64_t lora_workspace_bytes(int64_t M, int64_t R, int64_t K, int64_t E);
int64_t lora_max_rank();
void lora_shape(int64_t M, int64_t R, int64_t K, int64_t E, int *splits, int *shared);  // of a launch
bool lora_grid_ok(int64_t M, int64_t N, int64_t R, int64_t K, int64_t E);  // both launches fit a grid
hipError_t launch_lora_add(int type, const LoraArgs &a, hipStream_t s);

// ---- log probabilities of rows of logits (logprobs.hip); type is a qmm_float_type (of the logits).
struct LogprobArgs {
    const void *logits;     // row stride ld (elements)
    const uint32_t *mask;   // bit i of a row: token i is allowed; row stride mask_ld words (0: one row for all); or null
    const int32_t *tokens;  // [M][G]
    float *token_logprobs;  // [M][G]
    float *entropy;         // [M] or null
    int32_t *top_ids;       // [M][k]
    float *top_logprobs;    // [M][k]
    float4 *ws_stats;       // [M][splits], set by launch_logprobs
    uint64_t *ws_keys;      // [M][splits][k], set by launch_logprobs
    int64_t M, V, ld, mask_ld, G, k;
    float scale;
};
int64_t logprobs_max_k();
int logprobs_splits(int64_t M, int64_t V);  // workgroups per row
int64_t logprobs_max_rows();  // rows of one launch
int64_t logprobs_workspace_bytes(int64_t M, int64_t V, int64_t k);  // 0: not used
hipError_t launch_logprobs(int type, LogprobArgs a, void *ws, hipStream_t s);

// ---- rotary positions (rope.hip); type is a qmm_float_type (of x and out).
struct RopeArgs {
    const void *x;
    void *out;               // may be x
    const int32_t *positions;
    const float *factors;    // [rot / 2] or null
    int64_t ld_x, ld_out;    // elements from a token to the next
    int64_t head_x, head_out;  // elements from a head to the next
    int T, H, D, rot;
    double log2_base, freq_scale, low, high, magnitude;  // high <= low: no ramp
};
int64_t rope_max_dim();
hipError_t launch_rope(int type, bool interleaved, const RopeArgs &a, hipStream_t s);

// ---- the paged cache of 4-bit keys and values (kv_cache.hip, attention.hip, evict.hip)
struct KvCache {
    uint8_t *data;           // [pages][2][heads][page * D * 9 / 16]
    const int32_t *table;    // [B][width]
    const int32_t *lens;     // [B]
    const int32_t *starts;   // [B + 1] or null: one row each
    int pages, page_log2, heads, D, B, width, T;
};
hipError_t launch_cache_write(int type, const KvCache &c, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                              hipStream_t s);
hipError_t launch_cache_read(int type, const KvCache &c, void *k, void *v, hipStream_t s);

// attention of T rows of `group` query heads per cache head
struct AttendArgs {
    KvCache c;
    const void *q;           // [T][heads * group][D], ld_q elements from a row to the next
    void *out;               // likewise, ld_out
    float *lse;              // [T][heads * group] or null
    float *mass;             // [B][heads][ld_mass] or null
    float *ws;
    int64_t ld_q, ld_out, ld_mass;
    float scale;             // of the scores, times log2 e
    int group, window;       // window 0: none
    bool causal;
};
// of a call of up to T rows and B sequences; and what a call uses of it
int64_t attend_workspace_bytes(int type, int64_t T, int64_t B, int64_t capacity, int64_t heads, int64_t group, int64_t D,
                               bool ragged, bool mass);
int64_t attend_workspace_used(int type, const AttendArgs &a);
// splits of sequences with few rows, and with many (0: there can be none)
void attend_shape(int type, const AttendArgs &a, int *few, int *many);
bool attend_grid_ok(int type, const AttendArgs &a);  // every launch fits a grid
hipError_t launch_attend(int type, const AttendArgs &a, hipStream_t s);

// eviction: the entries that stay move from c.table's pages to those of `to`
struct EvictArgs {
    KvCache c;               // starts and T are not used
    const float *mass;       // [B][heads][ld_mass]
    const int32_t *to;       // [B][to_width]
    int32_t *lens_out;       // [B]
    float *mass_out;         // [B][heads][ld_out]
    int32_t *ids;            // [B][heads][budget]
    int64_t ld_mass, ld_out;
    int to_width, budget, recent;
};
// workgroups that move the entries into other pages
int64_t evict_workgroups(int64_t B, int64_t heads, int64_t D, int64_t capacity, int64_t budget);
hipError_t launch_cache_evict(const EvictArgs &a, hipStream_t s);

}  // namespace qmm
