// chunk.cuh -- launchers of the chunk operators (several new tokens per
// sequence into and over the paged cache), host arguments already checked.
#pragma once
#include "../../include/zdec.h"
#include "zdec_kernels.cuh"

namespace zdec {

// Sets the calling thread's global error message and returns s.
zdec_status fail_global(zdec_status s, const char *fmt, ...);

cudaError_t launch_chunk_plan(int R, const int32_t *ctx_len, const int32_t *n_new, const int32_t *free_pages,
                              int n_free, int32_t *tables, int max_pages, int T, int32_t *cu, int32_t *kv_len,
                              int32_t *positions, int64_t *slots, int32_t *taken, cudaStream_t stream);

struct RopeParams {
    unsigned long long turn[64];   // pair i: turns per position, 0.64 fixed point
    uint8_t axis[64];              // pair i: row of positions
    float4 table[64];              // (cos, sin) of i / 64 turns as hi + lo: cos hi, sin hi, cos lo, sin lo
};
struct ChunkAppendParams {
    KvPool kv;                     // base, page_bytes, n_pages, types, n_layers, n_kv (no table)
    int layer, T, nq, in_type, q_type;
    const void *qkv;
    long long ld, q_ld;
    const int32_t *positions;      // [axes][T]
    const int64_t *slots;
    void *q_out;
    uint32_t *status;
    int splits;                    // CTAs that share a token tile's query and key heads
    int tok_warp;                  // tokens of one warp of those
    int qk_ctas;                   // CTAs of queries and keys; the others move values
    int v_tile;                    // tokens of one of those
    RopeParams rope;
};
cudaError_t launch_chunk_append(ChunkAppendParams p, cudaStream_t stream);
cudaError_t launch_chunk_read(const KvPool &kv, int layer, int T, const int64_t *slots, uint16_t *k, uint16_t *v,
                              uint32_t *status, cudaStream_t stream);

struct ChunkAttnParams {
    KvPool kv;                     // table: [R][max_pages]
    int layer, nq, G, R, T, io_type, causal, window;
    int rows;                      // rows of an item: 128 or 256 (set by the launcher)
    float scale_log2;              // scale * log2(e)
    long long q_ld, o_ld;
    const int32_t *cu, *kv_len;
    const uint16_t *q;
    uint16_t *o;
    uint8_t *ws;
    uint32_t *status;
};
size_t chunk_attention_workspace(int nq, int nkv);
cudaError_t launch_chunk_attention(const ChunkAttnParams &p, cudaStream_t stream);

}  // namespace zdec
