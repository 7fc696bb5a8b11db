// chunk_api.cu -- C entries of the chunk operators: argument checks and
// launches (include/zdec.h, "chunks of new tokens").
#include <algorithm>
#include <array>
#include <initializer_list>
#include <cmath>

#include "chunk.cuh"

using namespace zdec;

#define CK(call)                                                                                   \
    do {                                                                                           \
        cudaError_t e_ = (call);                                                                   \
        if (e_ != cudaSuccess)                                                                     \
            return fail_global(ZDEC_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));     \
    } while (0)

namespace {
bool type_ok(int t) { return t == ZDEC_KV_F16 || t == ZDEC_KV_Q8_0 || t == ZDEC_KV_FP8; }
bool aligned16(const void *p) { return (uintptr_t)p % 16 == 0; }
constexpr int MAX_POOL_PAGES = 1 << 30, MAX_DIM = 1 << 16, MAX_R = 1 << 20, MAX_GROUP = 64;

zdec_status check_pool(const zdec_pool *pool, int layer) {
    if (!pool || !pool->base) return fail_global(ZDEC_ERR_ARG, "null pool");
    if (!aligned16(pool->base)) return fail_global(ZDEC_ERR_ARG, "the pool must be 16-byte aligned");
    if (!type_ok(pool->k_type) || !type_ok(pool->v_type)) return fail_global(ZDEC_ERR_ARG, "bad K or V cache type");
    if (pool->n_pages < 1 || pool->n_pages > MAX_POOL_PAGES || pool->n_layers < 1 || pool->n_layers > MAX_DIM ||
        pool->n_kv_heads < 1 || pool->n_kv_heads > MAX_DIM)
        return fail_global(ZDEC_ERR_ARG, "bad pool shape (%d pages, %d layers, %d kv heads)", pool->n_pages,
                           pool->n_layers, pool->n_kv_heads);
    if (layer < 0 || layer >= pool->n_layers)
        return fail_global(ZDEC_ERR_ARG, "layer %d outside [0, %d)", layer, pool->n_layers);
    return ZDEC_OK;
}
KvPool kv_of(const zdec_pool *pool, const int32_t *tables, int max_pages) {
    KvPool kv{};
    kv.base = (uint8_t *)pool->base;
    kv.page_bytes = zdec_page_bytes(pool->k_type, pool->v_type, pool->n_layers, pool->n_kv_heads);
    kv.n_pages = pool->n_pages;
    kv.k_type = pool->k_type;
    kv.v_type = pool->v_type;
    kv.n_layers = pool->n_layers;
    kv.n_kv = pool->n_kv_heads;
    kv.table = tables;
    kv.max_pages = max_pages;
    return kv;
}
// Whether two arrays, or T rows of wa and wb bytes that are la and lb bytes
// apart, share a byte.  Columns of one matrix (la == lb) may lie between each
// other; rows of different strides whose extents meet count as sharing.
bool overlap(const void *a, long long wa, const void *b, long long wb, long long T = 1, long long la = 0, long long lb = 0) {
    const __int128 x = (uintptr_t)a, y = (uintptr_t)b, d = y - x, rows = T - 1;
    if (!a || !b || wa <= 0 || wb <= 0 || x + rows * la + wa <= y || y + rows * lb + wb <= x) return false;
    if (la != lb || la == 0) return true;
    const long long in = (long long)(((d % la) + la) % la);   // where b's rows start within a's
    return in < wa || in + wb > la;
}
}  // namespace

extern "C" size_t zdec_page_bytes(int k_type, int v_type, int n_layers, int n_kv_heads) {
    if (!type_ok(k_type) || !type_ok(v_type) || n_layers < 1 || n_kv_heads < 1 || n_layers > MAX_DIM || n_kv_heads > MAX_DIM)
        return 0;
    return (size_t)n_layers * n_kv_heads * (kv_region_bytes(k_type) + kv_region_bytes(v_type));
}

extern "C" zdec_status zdec_chunk_plan(int R, const int32_t *ctx_len_dev, const int32_t *n_new_dev,
                                       const int32_t *free_pages_dev, int n_free, int32_t *tables_dev, int max_pages,
                                       int T, int32_t *cu_dev, int32_t *kv_len_dev, int32_t *positions_dev,
                                       int64_t *slots_dev, int32_t *taken_dev, void *stream) {
    if (R < 0 || R > MAX_R || T < 0) return fail_global(ZDEC_ERR_ARG, "R must be in [0, %d] and T >= 0", MAX_R);
    if (max_pages < 1 || max_pages > (1 << 25)) return fail_global(ZDEC_ERR_ARG, "max_pages must be in [1, %d]", 1 << 25);
    if (n_free < 0) return fail_global(ZDEC_ERR_ARG, "n_free must be >= 0");
    if (!cu_dev || !taken_dev || (R > 0 && (!ctx_len_dev || !n_new_dev || !tables_dev || !kv_len_dev)) ||
        (T > 0 && (!positions_dev || !slots_dev)))
        return fail_global(ZDEC_ERR_ARG, "null pointer");
    const long long r4 = 4LL * R;   // every CTA reads all lengths, at any time
    for (const int32_t *in : {ctx_len_dev, n_new_dev})
        if (overlap(in, r4, cu_dev, r4 + 4) || overlap(in, r4, kv_len_dev, r4) || overlap(in, r4, taken_dev, 8) ||
            overlap(in, r4, positions_dev, 4LL * T) || overlap(in, r4, slots_dev, 8LL * T))
            return fail_global(ZDEC_ERR_ARG, "an output overlaps ctx_len or n_new");
    CK(launch_chunk_plan(R, ctx_len_dev, n_new_dev, free_pages_dev, n_free, tables_dev, max_pages, T, cu_dev, kv_len_dev,
                         positions_dev, slots_dev, taken_dev, (cudaStream_t)stream));
    return ZDEC_OK;
}

extern "C" zdec_status zdec_chunk_append(const zdec_pool *pool, int layer, const zdec_rope *rope, int T, int n_q,
                                         const void *qkv_dev, int in_type, long long qkv_ld,
                                         const int32_t *positions_dev, const int64_t *slots_dev, void *q_out_dev,
                                         int q_type, long long q_ld, uint32_t *status_dev, void *stream) {
    zdec_status st = check_pool(pool, layer);
    if (st != ZDEC_OK) return st;
    if (!rope) return fail_global(ZDEC_ERR_ARG, "null rope");
    if (!(rope->theta >= 0.0f) || std::isinf(rope->theta)) return fail_global(ZDEC_ERR_ARG, "rope theta must be finite and >= 0");
    if (rope->axes < 1 || rope->axes > 4) return fail_global(ZDEC_ERR_ARG, "rope axes must be in [1, 4]");
    int pairs = 0;
    for (int a = 0; a < rope->axes; a++) {
        if (rope->sections[a] < 0 || rope->sections[a] > 64) return fail_global(ZDEC_ERR_ARG, "rope sections must be in [0, 64]");
        pairs += rope->sections[a];
    }
    if (pairs != 64) return fail_global(ZDEC_ERR_ARG, "rope sections sum to %d, not to 64 pairs", pairs);
    if (T < 0 || n_q < 0 || n_q > MAX_DIM) return fail_global(ZDEC_ERR_ARG, "bad T or n_q");
    if (in_type != ZDEC_F32 && in_type != ZDEC_F16 && in_type != ZDEC_BF16) return fail_global(ZDEC_ERR_ARG, "bad in_type");
    if (q_type != ZDEC_F16 && q_type != ZDEC_BF16) return fail_global(ZDEC_ERR_ARG, "q_type must be fp16 or bf16");
    if (T == 0) return ZDEC_OK;
    if (!qkv_dev || !positions_dev || !slots_dev || (n_q > 0 && !q_out_dev)) return fail_global(ZDEC_ERR_ARG, "null pointer");
    if (qkv_ld < (long long)(n_q + 2 * pool->n_kv_heads) * HD || qkv_ld % 8 || !aligned16(qkv_dev))
        return fail_global(ZDEC_ERR_ARG, "qkv rows must be 16-byte aligned, qkv_ld a multiple of 8 that holds n_q + 2 n_kv heads");
    if (n_q > 0 && (q_ld < (long long)n_q * HD || q_ld % 8 || !aligned16(q_out_dev)))
        return fail_global(ZDEC_ERR_ARG, "q rows must be 16-byte aligned, q_ld a multiple of 8 that holds n_q heads");
    const long long es = in_type == ZDEC_F32 ? 4 : 2;
    if (n_q > 0 && overlap(qkv_dev, (n_q + 2LL * pool->n_kv_heads) * HD * es, q_out_dev, 2LL * n_q * HD, T, qkv_ld * es, q_ld * 2))
        return fail_global(ZDEC_ERR_ARG, "q overlaps qkv");
    ChunkAppendParams p{};
    p.kv = kv_of(pool, nullptr, 0);
    p.layer = layer;
    p.T = T;
    p.nq = n_q;
    p.in_type = in_type;
    p.q_type = q_type;
    p.qkv = qkv_dev;
    p.ld = qkv_ld;
    p.q_ld = q_ld;
    p.positions = positions_dev;
    p.slots = slots_dev;
    p.q_out = q_out_dev;
    p.status = status_dev;
    static const std::array<float4, 64> table = [] {
        std::array<float4, 64> t;
        for (int i = 0; i < 64; i++) {
            const double c = std::cos(2.0 * M_PI * i / 64), s = std::sin(2.0 * M_PI * i / 64);
            t[i] = make_float4((float)c, (float)s, (float)(c - (float)c), (float)(s - (float)s));
        }
        return t;
    }();
    std::copy(table.begin(), table.end(), p.rope.table);
    // the fraction of a turn per position, as 0.64 fixed point: whole turns drop out (computed anew when theta changes)
    thread_local float known = -1.0f;
    thread_local unsigned long long turn[64];
    if (known != rope->theta) {
        for (int i = 0; i < 64; i++) {
            double t = rope->theta > 0.0f ? std::pow((double)rope->theta, -i / 64.0) / (2.0 * M_PI) : 0.0;
            t -= std::floor(t);
            turn[i] = (unsigned long long)std::ldexp(t, 64);
        }
        known = rope->theta;
    }
    std::copy(turn, turn + 64, p.rope.turn);
    int a = 0, left = rope->sections[0];
    for (int i = 0; i < 64; i++) {
        while (left == 0) left = rope->sections[++a];
        left--;
        p.rope.axis[i] = (uint8_t)a;
    }
    CK(launch_chunk_append(p, (cudaStream_t)stream));
    return ZDEC_OK;
}

extern "C" zdec_status zdec_chunk_read(const zdec_pool *pool, int layer, int T, const int64_t *slots_dev, void *k_dev,
                                       void *v_dev, uint32_t *status_dev, void *stream) {
    zdec_status st = check_pool(pool, layer);
    if (st != ZDEC_OK) return st;
    if (T < 0) return fail_global(ZDEC_ERR_ARG, "T must be >= 0");
    if (T == 0) return ZDEC_OK;
    if (!slots_dev || !k_dev || !v_dev) return fail_global(ZDEC_ERR_ARG, "null pointer");
    if (!aligned16(k_dev) || !aligned16(v_dev)) return fail_global(ZDEC_ERR_ARG, "k and v must be 16-byte aligned");
    CK(launch_chunk_read(kv_of(pool, nullptr, 0), layer, T, slots_dev, (uint16_t *)k_dev, (uint16_t *)v_dev, status_dev,
                         (cudaStream_t)stream));
    return ZDEC_OK;
}

extern "C" size_t zdec_chunk_attention_workspace_bytes(int n_q, int n_kv_heads) {
    if (n_q < 1 || n_kv_heads < 1 || n_q % n_kv_heads || n_q / n_kv_heads > MAX_GROUP) return 0;
    return chunk_attention_workspace(n_q, n_kv_heads);
}

extern "C" zdec_status zdec_chunk_attention(const zdec_pool *pool, int layer, const zdec_chunk_attn *a,
                                            const int32_t *cu_dev, const int32_t *kv_len_dev, const int32_t *tables_dev,
                                            const void *q_dev, void *o_dev, void *workspace_dev, size_t workspace_bytes,
                                            uint32_t *status_dev, void *stream) {
    zdec_status st = check_pool(pool, layer);
    if (st != ZDEC_OK) return st;
    if (!a) return fail_global(ZDEC_ERR_ARG, "null attention description");
    const int nkv = pool->n_kv_heads;
    if (a->n_q < 1 || a->n_q % nkv) return fail_global(ZDEC_ERR_ARG, "n_q must be a multiple of n_kv_heads");
    if (a->n_q / nkv > MAX_GROUP) return fail_global(ZDEC_ERR_UNSUPPORTED, "at most %d query heads per kv head", MAX_GROUP);
    if (a->R < 0 || a->R > MAX_R || a->T < 0) return fail_global(ZDEC_ERR_ARG, "R must be in [0, %d] and T >= 0", MAX_R);
    if ((long long)a->T * a->n_q > 0x7FFFFFFFLL) return fail_global(ZDEC_ERR_UNSUPPORTED, "T * n_q must stay below 2^31");
    if (a->max_pages < 1 || a->max_pages > (1 << 25)) return fail_global(ZDEC_ERR_ARG, "max_pages must be in [1, %d]", 1 << 25);
    if (a->io_type != ZDEC_F16 && a->io_type != ZDEC_BF16) return fail_global(ZDEC_ERR_ARG, "q and o are fp16 or bf16");
    if (a->window < 0 || (a->window > 0 && !a->causal)) return fail_global(ZDEC_ERR_ARG, "a window must be >= 0 and needs the causal mask");
    if (!(a->scale > 0.0f) || std::isinf(a->scale)) return fail_global(ZDEC_ERR_ARG, "scale must be finite and > 0");
    if (a->R == 0 || a->T == 0) return ZDEC_OK;
    if (!cu_dev || !kv_len_dev || !tables_dev || !q_dev || !o_dev) return fail_global(ZDEC_ERR_ARG, "null pointer");
    const long long need = (long long)a->n_q * HD;
    if (a->q_ld < need || a->q_ld % 8 || a->o_ld < need || a->o_ld % 8 || !aligned16(q_dev) || !aligned16(o_dev))
        return fail_global(ZDEC_ERR_ARG, "q and o rows must be 16-byte aligned, their strides multiples of 8 that hold n_q heads");
    if (!workspace_dev || (uintptr_t)workspace_dev % 256) return fail_global(ZDEC_ERR_ARG, "the workspace must be 256-byte aligned");
    if (workspace_bytes < zdec_chunk_attention_workspace_bytes(a->n_q, nkv)) return fail_global(ZDEC_ERR_ARG, "workspace too small");
    if (overlap(q_dev, need * 2, o_dev, need * 2, a->T, a->q_ld * 2, a->o_ld * 2)) return fail_global(ZDEC_ERR_ARG, "o overlaps q");
    ChunkAttnParams p{};
    p.kv = kv_of(pool, tables_dev, a->max_pages);
    p.layer = layer;
    p.nq = a->n_q;
    p.G = a->n_q / nkv;
    p.R = a->R;
    p.T = a->T;
    p.io_type = a->io_type;
    p.causal = a->causal != 0;
    p.window = a->window;
    p.scale_log2 = (float)((double)a->scale * 1.4426950408889634);
    p.q_ld = a->q_ld;
    p.o_ld = a->o_ld;
    p.cu = cu_dev;
    p.kv_len = kv_len_dev;
    p.q = (const uint16_t *)q_dev;
    p.o = (uint16_t *)o_dev;
    p.ws = (uint8_t *)workspace_dev;
    p.status = status_dev;
    CK(launch_chunk_attention(p, (cudaStream_t)stream));
    return ZDEC_OK;
}
