// chunk.cu -- a chunk of new tokens into the paged cache: the plan of a
// ragged batch, the append and the read-back.
#include "chunk.cuh"

namespace zdec {

constexpr uint32_t FULL = 0xFFFFFFFFu;

// ------------------------------------------------------------------ plan ---
// One launch.  Every CTA scans the requests' (new tokens, new pages) on its
// own, in strips of one request per thread (8 bytes each, from L2 after the
// first CTA), and resolves its own tokens by binary search in the strip: no
// CTA waits for another, and the only large traffic is the 12 bytes per token
// written.  A new page is set by the token at its first position, which is
// always one of the new tokens.  32 requests of one token: 4.7 us, 1024 prompts
// of 966000 tokens: 11.8 us (the bytes: 1.7); launch, one strip's scan and the
// chain ctx_len -> table entry -> slot are what it takes.
constexpr int PLAN_THREADS = 512, PLAN_TOK = 4;   // threads (= requests per strip), tokens per thread

__global__ __launch_bounds__(PLAN_THREADS) void plan_kernel(int R, const int32_t *__restrict__ ctx_len,
                                                            const int32_t *__restrict__ n_new,
                                                            const int32_t *__restrict__ free_pages, int n_free,
                                                            int32_t *tables, int max_pages, int T, int32_t *cu,
                                                            int32_t *kv_len, int32_t *positions, int64_t *slots,
                                                            int32_t *taken) {
    __shared__ uint32_t s_tok[PLAN_THREADS], s_page[PLAN_THREADS];   // exclusive sums within the strip
    __shared__ int32_t s_ctx[PLAN_THREADS];
    __shared__ unsigned long long s_warp[PLAN_THREADS / 32], s_tot;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long t0 = ((long long)blockIdx.x * PLAN_THREADS + tid) * PLAN_TOK;
    const long long cta_end = ((long long)blockIdx.x + 1) * PLAN_THREADS * PLAN_TOK;
    int32_t pos[PLAN_TOK];
    int64_t slot[PLAN_TOK];
#pragma unroll
    for (int i = 0; i < PLAN_TOK; i++) { pos[i] = -1; slot[i] = -1; }
    uint32_t tok_base = 0, page_base = 0;   // sums of the strips before
    const bool writer = blockIdx.x == 0;
    for (int r0 = 0; r0 < R; r0 += PLAN_THREADS) {
        const int r = r0 + tid;
        const int c = r < R ? max(0, ctx_len[r]) : 0, n = r < R ? max(0, n_new[r]) : 0;
        const int held = (int)min((long long)max_pages, ((long long)c + 63) / 64);
        const int need = (int)min((long long)max_pages, ((long long)c + n + 63) / 64);
        // tokens in the low word, pages in the high one: sums below 2^31 do not carry
        const unsigned long long own = (unsigned long long)(uint32_t)n | ((unsigned long long)(uint32_t)(need - held) << 32);
        unsigned long long incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const unsigned long long w = lane < PLAN_THREADS / 32 ? s_warp[lane] : 0;
            unsigned long long wi = w;
#pragma unroll
            for (int o = 1; o < PLAN_THREADS / 32; o <<= 1) {
                const unsigned long long v = __shfl_up_sync(FULL, wi, o);
                if (lane >= o) wi += v;
            }
            if (lane < PLAN_THREADS / 32) s_warp[lane] = wi - w;
            if (lane == PLAN_THREADS / 32 - 1) s_tot = wi;
        }
        __syncthreads();
        const unsigned long long excl = incl - own + s_warp[warp];
        s_tok[tid] = (uint32_t)excl;
        s_page[tid] = (uint32_t)(excl >> 32);
        s_ctx[tid] = c;
        if (writer && r < R) {
            cu[r] = (int32_t)(tok_base + (uint32_t)excl);
            kv_len[r] = (int32_t)min(0x7FFFFFFFLL, (long long)c + n);
        }
        const uint32_t strip_tok = (uint32_t)s_tot, strip_page = (uint32_t)(s_tot >> 32);
        __syncthreads();
        const long long lo = tok_base, hi = lo + strip_tok;
        if (hi > t0 && lo < t0 + PLAN_TOK) {
            int at = -1;   // the strip's request of the current token
            uint32_t next = 0;
#pragma unroll
            for (int i = 0; i < PLAN_TOK; i++) {
                const long long t = t0 + i;
                if (t >= T || t < lo || t >= hi) continue;
                const uint32_t x = (uint32_t)(t - lo);
                if (at < 0 || x >= next) {   // the last request that starts at or before x
                    int a = 0, b = min(PLAN_THREADS, R - r0);
                    while (b - a > 1) {
                        const int m = (a + b) >> 1;
                        if (s_tok[m] <= x) a = m;
                        else b = m;
                    }
                    at = a;
                    next = a + 1 < min(PLAN_THREADS, R - r0) ? s_tok[a + 1] : strip_tok;
                }
                const int cc = s_ctx[at];
                const long long p64 = (long long)cc + (x - s_tok[at]);
                pos[i] = (int32_t)min(0x7FFFFFFFLL, p64);
                const long long pg = p64 >> 6;
                if (pg < max_pages) {
                    const int first = (int)(((long long)cc + 63) >> 6);
                    int32_t *entry = tables + (size_t)(r0 + at) * max_pages + pg;
                    int page;
                    if (free_pages && pg >= first) {
                        const long long f = (long long)page_base + s_page[at] + (pg - first);
                        page = f < n_free ? free_pages[f] : -1;
                        if ((p64 & 63) == 0) *entry = page;
                    } else {
                        page = *entry;
                    }
                    if (page >= 0) slot[i] = (int64_t)page * 64 + (p64 & 63);
                }
            }
        }
        tok_base += strip_tok;
        page_base += strip_page;
        __syncthreads();
        if (!writer && (long long)tok_base >= cta_end) break;   // the same on every thread
    }
    if (writer && tid == 0) {
        cu[R] = (int32_t)tok_base;
        taken[0] = (int32_t)page_base;
        taken[1] = (int32_t)tok_base;
    }
    if (t0 + PLAN_TOK <= T && ((uintptr_t)positions % 16) == 0 && ((uintptr_t)slots % 16) == 0) {
        *reinterpret_cast<int4 *>(positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<longlong2 *>(slots + t0) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2 *>(slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
        for (int i = 0; i < PLAN_TOK; i++)
            if (t0 + i < T) {
                positions[t0 + i] = pos[i];
                slots[t0 + i] = slot[i];
            }
    }
}

cudaError_t launch_chunk_plan(int R, const int32_t *ctx_len, const int32_t *n_new, const int32_t *free_pages,
                              int n_free, int32_t *tables, int max_pages, int T, int32_t *cu, int32_t *kv_len,
                              int32_t *positions, int64_t *slots, int32_t *taken, cudaStream_t stream) {
    const long long per = PLAN_THREADS * PLAN_TOK;
    const unsigned grid = (unsigned)std::max(1LL, ((long long)T + per - 1) / per);
    plan_kernel<<<grid, PLAN_THREADS, 0, stream>>>(R, ctx_len, n_new, free_pages, n_free, tables, max_pages, T, cu, kv_len,
                                                   positions, slots, taken);
    return cudaGetLastError();
}

// ------------------------------------------------------- page addressing ---
__device__ __forceinline__ uint8_t *chunk_of_page(const KvPool &p, int layer, int head, long long page) {
    return p.base + (size_t)page * p.page_bytes + kv_chunk_off(p, layer, head);
}
// A token's slot as (page, token within it): -1 without one; a slot past the
// pool counts as none and is reported.
__device__ __forceinline__ long long checked_slot(const KvPool &p, long long slot, uint32_t *status) {
    if (slot < 0) return -1;
    if ((slot >> 6) >= p.n_pages) {
        if (status) atomicOr(status, (uint32_t)ZDEC_CHUNK_BAD_SLOT);
        return -1;
    }
    return slot;
}

// ---------------------------------------------------------------- append ---
// Eight consecutive elements of a row as fp32.
template <int IN>
__device__ __forceinline__ void load8(const void *p, long long i, float (&x)[8]) {
    if (IN == ZDEC_F32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = __ldcs(q), b = __ldcs(q + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float2 f = IN == ZDEC_F16 ? __half22float2(u32_as_h2(w[k]))
                                            : make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
            x[2 * k] = f.x;
            x[2 * k + 1] = f.y;
        }
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {   // nearest even, low half x
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) { return h2_as_u32(__floats2half2_rn(x, y)); }

// Two fp16 values -> two stored bytes (low first): e4m3, or Q8_0 codes + 128
// of a block with fp32 scale d (0 for an all-zero block).
__device__ __forceinline__ uint32_t fp8_pair(uint32_t h2) {
    uint16_t out;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(out) : "r"(h2));
    return out;
}
__device__ __forceinline__ uint32_t q8_code(float x, float d) {
    if (d == 0.0f) return 128u;
    const int q = max(-127, min(127, __float2int_rn(__fdiv_rn(x, d))));
    return (uint32_t)(q + 128) & 0xFFu;
}
// Eight of them.  x times the reciprocal lies within 1e-4 of the rounded
// quotient (127 x 7 2^-24), so where it is not within that of a half, both
// round to the same integer, read off a sum with 1.5 2^23 + 128; else (and for
// what is not finite) the eight are divided.
__device__ __forceinline__ uint2 q8_codes(const float (&f)[8], float d) {
    const float inv = d == 0.0f ? 0.0f : __fdividef(1.0f, d);
    uint32_t c[2], t[8];
    bool near = true;
#pragma unroll
    for (int k = 0; k < 8; k++) {
        const float r = __fmul_rn(f[k], inv), s = __fadd_rn(r, 12583040.0f);
        near = near && fabsf(r - __fadd_rn(s, -12583040.0f)) < 0.4999f;
        t[k] = __float_as_uint(s);
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
        c[i] = __byte_perm(__byte_perm(t[4 * i], t[4 * i + 1], 0x0040), __byte_perm(t[4 * i + 2], t[4 * i + 3], 0x0040), 0x5410);
    if (!near) {
        c[0] = c[1] = 0u;
#pragma unroll
        for (int k = 0; k < 8; k++) c[k >> 2] |= q8_code(f[k], d) << (8 * (k & 3));
    }
    return make_uint2(c[0], c[1]);
}
// A block's scale from its amax: fp32 IEEE division (0 for an all-zero block).
__device__ __forceinline__ float q8_scale(float amax) { return amax == 0.0f ? 0.0f : __fdiv_rn(amax, 127.0f); }

// Eight fp32 in storage form: fp16 (16 bytes) or codes (8 bytes), a Q8_0
// block's 32 dims being held by 4 neighbouring lanes.
template <int T>
__device__ __forceinline__ uint4 encode8(const float (&x)[8], float &scale) {
    uint4 h = make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]), pack_f16(x[6], x[7]));
    if (T == KV_T_F16) return h;
    if (T == KV_T_FP8) return make_uint4(fp8_pair(h.x) | (fp8_pair(h.y) << 16), fp8_pair(h.z) | (fp8_pair(h.w) << 16), 0u, 0u);
    const uint32_t w[4] = {h.x, h.y, h.z, h.w};
    float f[8], m = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float2 v = __half22float2(u32_as_h2(w[k]));
        f[2 * k] = v.x;
        f[2 * k + 1] = v.y;
        m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
    m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
    m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
    scale = q8_scale(m);
    const uint2 c = q8_codes(f, scale);
    return make_uint4(c.x, c.y, 0u, 0u);
}

constexpr int AP_THREADS = 256, AP_WARPS = AP_THREADS / 32, AP_TILE = 64;   // AP_TILE: most tokens of a value-head CTA
// Tokens of a CTA that moves one head's values: 64, or 16 where that leaves SMs without a CTA (77 tokens of 8 heads
// read back: 8.0 us with 64, 3.9 with 16).
static int value_tile(long long T, int n_kv) { return (T + AP_TILE - 1) / AP_TILE * n_kv < 152 ? 16 : AP_TILE; }

// cos and sin of position x turns (0.64 fixed point), nearly rounded to
// nearest: the nearest 64th of a turn from the table (hi + lo), the rest, at
// most 2 pi / 128, by the Taylor series, joined by the addition theorems with
// only the last sum rounded at full size (error below 2^-24.9).
__device__ __forceinline__ float2 turn_cos_sin(unsigned long long x, const float4 *table) {
    const unsigned long long k = (x + (1ULL << 57)) >> 58;
    const float r = (float)(int)((long long)(x - (k << 58)) >> 27) * 4.5716142e-11f;   // 2 pi 2^-37
    const float4 t = table[k & 63];
    const float r2 = r * r;
    const float s = fmaf(r * r2, fmaf(r2, 1.0f / 120.0f, -1.0f / 6.0f), r);            // sin r
    const float c = r2 * fmaf(r2, fmaf(r2, -1.0f / 720.0f, 1.0f / 24.0f), -0.5f);      // cos r - 1
    return make_float2(t.x + (fmaf(t.x, c, -t.y * s) + t.z), t.y + (fmaf(t.y, c, t.x * s) + t.w));
}

// Bounded by HBM for long prompts (18600 tokens, 32 + 8 + 8 heads, bf16
// into FP8: 419 MB in 83 us, 5.0 TB/s, 75 % of the copy rate; the table lookups'
// arithmetic and the fp32 products fill much of the issue slots), by latency for
// short ones (8 tokens: 4.1 us).
//
// Rotation of the query and key heads.  A warp takes a token's heads four at
// a time: 8 lanes per head, lane j the pairs 8j .. 8j + 7 (dims 8j.. and
// 64 + 8j..: 16-byte loads and stores).  The 64 angles are computed once per
// token, two per lane, and passed through shared memory.
template <int IN, int KT>
__device__ __forceinline__ void append_qk(const ChunkAppendParams &p, long long tile, int split, const unsigned long long *s_turn,
                                          const uint8_t *s_axis, const float4 *s_table, float2 (*s_cs)[64]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane & 7;
    const int heads = p.nq + p.kv.n_kv, groups = (heads + 3) / 4;
    const int g0 = (int)((long long)groups * split / p.splits), g1 = (int)((long long)groups * (split + 1) / p.splits);
    for (int i = 0; i < p.tok_warp; i++) {
        const long long t = (tile * p.tok_warp + i) * AP_WARPS + warp;
        if (t >= p.T) break;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int pair = lane + 32 * k;
            const long long pos = __ldg(p.positions + (size_t)s_axis[pair] * p.T + t);
            s_cs[warp][pair] = turn_cos_sin((unsigned long long)pos * s_turn[pair], s_table);
        }
        const long long slot = checked_slot(p.kv, __ldg(p.slots + t), p.status);
        __syncwarp();
        float2 cs[8];
#pragma unroll
        for (int k = 0; k < 8; k++) cs[k] = s_cs[warp][8 * j + k];
        const long long row = t * p.ld;
#pragma unroll 2
        for (int g = g0; g < g1; g++) {
            const int h = 4 * g + (lane >> 3), hh = min(h, heads - 1);   // lanes past the last head repeat it
            float a[8], b[8], x[8], y[8];
            load8<IN>(p.qkv, row + (long long)hh * HD + 8 * j, a);
            load8<IN>(p.qkv, row + (long long)hh * HD + 64 + 8 * j, b);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                // a c - b s and b c + a s with the second product's rounding error put back
                const float u = b[k] * cs[k].y, v = a[k] * cs[k].y;
                x[k] = fmaf(a[k], cs[k].x, -u) - fmaf(b[k], cs[k].y, -u);
                y[k] = fmaf(b[k], cs[k].x, v) + fmaf(a[k], cs[k].y, -v);
            }
            if (h < p.nq) {
                uint4 *q = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.q_out) + t * p.q_ld + (long long)h * HD + 8 * j);
                if (p.q_type == ZDEC_F16) {
                    q[0] = make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]), pack_f16(x[6], x[7]));
                    q[8] = make_uint4(pack_f16(y[0], y[1]), pack_f16(y[2], y[3]), pack_f16(y[4], y[5]), pack_f16(y[6], y[7]));
                } else {
                    q[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                    q[8] = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
                }
            }
            if (4 * g + 3 < p.nq) continue;   // no key head in this group
            float dx = 0.0f, dy = 0.0f;
            const uint4 ex = encode8<KT>(x, dx), ey = encode8<KT>(y, dy);
            if (slot < 0 || h < p.nq || h >= heads) continue;
            uint8_t *reg = chunk_of_page(p.kv, p.layer, h - p.nq, slot >> 6);
            const int tl = (int)(slot & 63);
            if (KT == KV_T_F16) {
                *reinterpret_cast<uint4 *>(reg + k16_off(tl, 8 * j)) = ex;
                *reinterpret_cast<uint4 *>(reg + k16_off(tl, 64 + 8 * j)) = ey;
            } else {
                *reinterpret_cast<uint2 *>(reg + k8_off(tl, 8 * j)) = make_uint2(ex.x, ex.y);
                *reinterpret_cast<uint2 *>(reg + k8_off(tl, 64 + 8 * j)) = make_uint2(ey.x, ey.y);
                if (KT == KV_T_Q8 && (j & 3) == 0) {
                    *reinterpret_cast<uint16_t *>(reg + ks_off(tl, j >> 2)) = __half_as_ushort(__float2half_rn(dx));
                    *reinterpret_cast<uint16_t *>(reg + ks_off(tl, 2 + (j >> 2))) = __half_as_ushort(__float2half_rn(dy));
                }
            }
        }
    }
}

// What a tile's tokens do with the 16-byte value segments of `seg` tokens: 1
// the token opens a segment that the tile fills, 0 it lies inside one, 2 its
// element goes alone, 3 it has no slot.  Threads 0 to 63 ask, one token each;
// `todo` gets a bit per token that is not 0.
__device__ __forceinline__ void segment_roles(const long long *s_slot, int n, int seg, uint8_t *role, uint32_t *todo) {
    const int i = threadIdx.x;
    if (i >= AP_TILE) return;
    int r = 0;
    if (i < n) {
        const long long slot = s_slot[i];
        const int in = (int)(slot & (seg - 1)), a = i - in;   // a: where the segment's first token would be
        r = slot < 0 ? 3 : a < 0 || a + seg > n ? 2 : in == 0;
        if (r < 2) {
            bool whole = true;
#pragma unroll 8
            for (int e = 0; e < seg; e++) whole = whole && s_slot[a + e] == slot - in + e;
            if (!whole) r = 2;
        }
        role[i] = (uint8_t)r;
    }
    const uint32_t bits = __ballot_sync(FULL, r != 0);
    if ((i & 31) == 0) todo[i >> 5] = bits;
}
// The bits of tokens lo .. lo + len - 1 (len <= 32), lo a multiple of len.
__device__ __forceinline__ uint32_t todo_of(const uint32_t *todo, int lo, int len) {
    const uint32_t w = todo[lo >> 5] >> (lo & 31);
    return len == 32 ? w : w & ((1u << len) - 1);
}

// One value head of up to AP_TILE tokens: encoded rows meet in shared memory
// and leave transposed, 16 bytes (8 or 16 tokens of one dim) at a time where
// those tokens fill one 16-byte segment of the page, else element by element.
template <int IN, int VT>
__device__ __forceinline__ void append_v(const ChunkAppendParams &p, long long tile, int head, uint8_t *smem, long long *s_slot,
                                         uint8_t *s_role, uint32_t *s_todo) {
    constexpr int ES = VT == KV_T_F16 ? 2 : 1, SEG = 16 / ES;
    constexpr int PITCH = HD * ES + 16;   // bytes of a row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane & 15;
    const long long t0 = tile * p.v_tile;
    const int n = (int)min((long long)p.v_tile, p.T - t0);
    if ((int)threadIdx.x < n) s_slot[threadIdx.x] = checked_slot(p.kv, __ldg(p.slots + t0 + threadIdx.x), p.status);
    __syncthreads();
    segment_roles(s_slot, n, SEG, s_role, s_todo);
    const long long col = (long long)(p.nq + p.kv.n_kv + head) * HD;
#pragma unroll 2
    for (int i0 = 2 * warp; i0 < n; i0 += 2 * AP_WARPS) {   // two tokens of 16 lanes x 8 dims
        const int i = i0 + (lane >> 4), ii = min(i, n - 1);
        float x[8], d = 0.0f;
        load8<IN>(p.qkv, (t0 + ii) * p.ld + col + 8 * j, x);
        const uint4 e = encode8<VT>(x, d);
        if (i >= n) continue;
        if (VT == KV_T_F16) *reinterpret_cast<uint4 *>(smem + i * PITCH + 16 * j) = e;
        else *reinterpret_cast<uint2 *>(smem + i * PITCH + 8 * j) = make_uint2(e.x, e.y);
        const long long slot = s_slot[i];
        if (VT == KV_T_Q8 && (j & 3) == 0 && slot >= 0) {
            uint8_t *reg = chunk_of_page(p.kv, p.layer, head, slot >> 6) + kv_region_bytes(p.kv.k_type);
            *reinterpret_cast<uint16_t *>(reg + vs_off((int)(slot & 63), j >> 2)) = __half_as_ushort(__float2half_rn(d));
        }
    }
    __syncthreads();
    // thread = dim and half of the tokens
    const int d = threadIdx.x & (HD - 1), half = p.v_tile / 2, first = (threadIdx.x >> 7) * half;
    for (uint32_t bits = todo_of(s_todo, first, half); bits; bits &= bits - 1) {
        const int i = first + __ffs(bits) - 1, role = s_role[i];
        if (role == 3) continue;
        const long long slot = s_slot[i];
        uint8_t *reg = chunk_of_page(p.kv, p.layer, head, slot >> 6) + kv_region_bytes(p.kv.k_type);
        const int tl = (int)(slot & 63);
        uint8_t *dst = reg + (VT == KV_T_F16 ? v16_off(tl, d) : v8_off(tl, d));
        const uint8_t *src = smem + i * PITCH + d * ES;
        if (role == 1) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; e++)
                w[e] = ES == 2 ? (uint32_t)*reinterpret_cast<const uint16_t *>(src + (2 * e) * PITCH) |
                                     ((uint32_t)*reinterpret_cast<const uint16_t *>(src + (2 * e + 1) * PITCH) << 16)
                               : (uint32_t)src[(4 * e) * PITCH] | ((uint32_t)src[(4 * e + 1) * PITCH] << 8) |
                                     ((uint32_t)src[(4 * e + 2) * PITCH] << 16) | ((uint32_t)src[(4 * e + 3) * PITCH] << 24);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if (ES == 2) {
            *reinterpret_cast<uint16_t *>(dst) = *reinterpret_cast<const uint16_t *>(src);
        } else {
            *dst = *src;
        }
    }
}

template <int IN>
__global__ __launch_bounds__(AP_THREADS) void chunk_append_kernel(const __grid_constant__ ChunkAppendParams p) {
    union Shared {
        struct { unsigned long long turn[64]; float4 table[64]; float2 cs[AP_WARPS][64]; uint8_t axis[64]; } qk;
        struct { uint8_t v[AP_TILE * (HD * 2 + 16)]; long long slot[AP_TILE]; uint8_t role[AP_TILE]; uint32_t todo[2]; } v;
    };
    __shared__ __align__(16) Shared s;
    if ((int)blockIdx.x < p.qk_ctas) {
        if (threadIdx.x < 64) {
            s.qk.turn[threadIdx.x] = p.rope.turn[threadIdx.x];
            s.qk.table[threadIdx.x] = p.rope.table[threadIdx.x];
            s.qk.axis[threadIdx.x] = p.rope.axis[threadIdx.x];
        }
        __syncthreads();
        const long long tile = blockIdx.x / p.splits;
        const int split = blockIdx.x % p.splits;
        switch (p.kv.k_type) {
            case KV_T_F16: append_qk<IN, KV_T_F16>(p, tile, split, s.qk.turn, s.qk.axis, s.qk.table, s.qk.cs); break;
            case KV_T_Q8: append_qk<IN, KV_T_Q8>(p, tile, split, s.qk.turn, s.qk.axis, s.qk.table, s.qk.cs); break;
            default: append_qk<IN, KV_T_FP8>(p, tile, split, s.qk.turn, s.qk.axis, s.qk.table, s.qk.cs); break;
        }
    } else {
        const unsigned v = blockIdx.x - p.qk_ctas;
        const long long tile = v / p.kv.n_kv;
        const int head = v % p.kv.n_kv;
        switch (p.kv.v_type) {
            case KV_T_F16: append_v<IN, KV_T_F16>(p, tile, head, s.v.v, s.v.slot, s.v.role, s.v.todo); break;
            case KV_T_Q8: append_v<IN, KV_T_Q8>(p, tile, head, s.v.v, s.v.slot, s.v.role, s.v.todo); break;
            default: append_v<IN, KV_T_FP8>(p, tile, head, s.v.v, s.v.slot, s.v.role, s.v.todo); break;
        }
    }
}

cudaError_t launch_chunk_append(ChunkAppendParams p, cudaStream_t stream) {
    const int groups = (p.nq + p.kv.n_kv + 3) / 4;
    // Few tokens: their heads are split until a wave of CTAs is full; many: a warp takes two tokens, which halves the
    // CTAs' start (tables into shared memory; 5000 tokens 22.4 us with two, 23.3 with one, 2500 26.4 and 20.6).
    p.tok_warp = p.T > 4 * 152 * AP_WARPS ? 2 : 1;
    const long long tiles = ((long long)p.T + AP_WARPS * p.tok_warp - 1) / (AP_WARPS * p.tok_warp);
    p.splits = (int)std::max(1LL, std::min((long long)groups, 2 * 152 / tiles));
    p.v_tile = value_tile(p.T, p.kv.n_kv);
    const long long qk = tiles * p.splits, v = ((long long)p.T + p.v_tile - 1) / p.v_tile * p.kv.n_kv;
    if (qk + v > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    p.qk_ctas = (int)qk;
    const unsigned grid = (unsigned)(qk + v);
    switch (p.in_type) {
        case ZDEC_F32: chunk_append_kernel<ZDEC_F32><<<grid, AP_THREADS, 0, stream>>>(p); break;
        case ZDEC_F16: chunk_append_kernel<ZDEC_F16><<<grid, AP_THREADS, 0, stream>>>(p); break;
        default: chunk_append_kernel<ZDEC_BF16><<<grid, AP_THREADS, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

// ------------------------------------------------------------------ read ---
// Two stored values (the bytes of `c` that `sel` picks, as __byte_perm does
// with 0x64 as byte 4) as fp16: for Q8_0 1024 + code read as fp16, less 1152,
// times the scale (the product of 8 and 11 bits, rounded once), at most fp16's
// largest value (127 x a scale of 516 lies past it; `big`: a scale above 511).
__device__ __forceinline__ uint32_t q8_pair(uint32_t c, uint32_t sel, uint32_t scale2, bool big) {
    __half2 x = __hmul2(__hsub2(u32_as_h2(__byte_perm(c, 0x64u, sel)), u32_as_h2(0x64806480u)), u32_as_h2(scale2));
    if (big) x = __hmax2_nan(__hmin2_nan(x, u32_as_h2(0x7BFF7BFFu)), u32_as_h2(0xFBFFFBFFu));
    return h2_as_u32(x);
}
__device__ __forceinline__ bool big_scale(uint32_t bits) { return (bits & 0x7FFFu) > 0x5FFCu; }   // above 511, or not finite
// Eight codes -> eight fp16.
template <int T>
__device__ __forceinline__ uint4 decode8(uint2 c, uint32_t scale) {
    if (T == KV_T_FP8)
        return make_uint4(e4m3x2_to_h2((uint16_t)c.x), e4m3x2_to_h2((uint16_t)(c.x >> 16)), e4m3x2_to_h2((uint16_t)c.y),
                          e4m3x2_to_h2((uint16_t)(c.y >> 16)));
    const uint32_t s2 = scale * 0x10001u;
    const bool big = big_scale(scale);
    return make_uint4(q8_pair(c.x, 0x4140, s2, big), q8_pair(c.x, 0x4342, s2, big), q8_pair(c.y, 0x4140, s2, big),
                      q8_pair(c.y, 0x4342, s2, big));
}

// A CTA reads one kv head of up to AP_TILE slots.  K rows go straight through
// registers; V goes through shared memory, a 16-byte segment (8
// or 16 tokens of one dim) at a time where the tile's slots fill it: a thread
// takes two dims and a quarter of the tokens, the lane halves of a warp
// neighbouring quarters (whole 32-byte sectors), and puts the two dims down
// as one word, columns swapped so that the lane halves' rows, 16 apart, do not
// meet in a bank.  30000 Q8_0 tokens of 8 heads (188 MB): 36 us, 5.2 TB/s, 78 %
// of the copy rate; a thread per dim and scalar decoding took 55 us.  77 tokens:
// 4 us.
template <int KT, int VT>
__global__ __launch_bounds__(AP_THREADS) void chunk_read_kernel(const __grid_constant__ KvPool a, int layer, int T, int tile,
                                                                const int64_t *__restrict__ slots, uint16_t *__restrict__ k,
                                                                uint16_t *__restrict__ v, uint32_t *status) {
    constexpr int SEG = VT == KV_T_F16 ? 8 : 16;
    __shared__ __align__(16) uint32_t s_v[AP_TILE * HD / 2];
    __shared__ long long s_slot[AP_TILE];
    __shared__ uint32_t s_todo[2];
    __shared__ uint32_t s_scale[AP_TILE][4];   // a block's scale, twice
    __shared__ uint8_t s_role[AP_TILE];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane & 15;
    const long long t0 = (long long)(blockIdx.x / a.n_kv) * tile;
    const int head = blockIdx.x % a.n_kv, n = (int)min((long long)tile, T - t0);
    if ((int)threadIdx.x < n) s_slot[threadIdx.x] = checked_slot(a, __ldg(slots + t0 + threadIdx.x), status);
    __syncthreads();
    // K's rows on their way first: two tokens of 16 lanes x 8 dims per warp
    uint4 kx[AP_TILE / (2 * AP_WARPS)];
    uint32_t ks[AP_TILE / (2 * AP_WARPS)];
#pragma unroll
    for (int m = 0; m < AP_TILE / (2 * AP_WARPS); m++) {
        const int i = 2 * (warp + m * AP_WARPS) + (lane >> 4);
        const long long slot = i < n ? s_slot[i] : -1;
        kx[m] = make_uint4(0u, 0u, 0u, 0u);
        ks[m] = 0u;
        if (slot < 0) {
            if (KT == KV_T_Q8) kx[m].x = kx[m].y = 0x80808080u;
            continue;
        }
        const uint8_t *reg = chunk_of_page(a, layer, head, slot >> 6);
        const int tl = (int)(slot & 63);
        if (KT == KV_T_F16) {
            kx[m] = *reinterpret_cast<const uint4 *>(reg + k16_off(tl, 8 * j));
        } else {
            const uint2 c = *reinterpret_cast<const uint2 *>(reg + k8_off(tl, 8 * j));
            kx[m].x = c.x;
            kx[m].y = c.y;
            if (KT == KV_T_Q8) ks[m] = *reinterpret_cast<const uint16_t *>(reg + ks_off(tl, j >> 2));
        }
    }
    segment_roles(s_slot, n, SEG, s_role, s_todo);
    bool big = false;
    if (VT == KV_T_Q8 && (int)threadIdx.x < 4 * n) {
        const long long slot = s_slot[threadIdx.x >> 2];
        if (slot >= 0) {
            const uint32_t s = *reinterpret_cast<const uint16_t *>(chunk_of_page(a, layer, head, slot >> 6) +
                                                                   kv_region_bytes(a.k_type) +
                                                                   vs_off((int)(slot & 63), threadIdx.x & 3));
            s_scale[threadIdx.x >> 2][threadIdx.x & 3] = s * 0x10001u;
            big = big_scale(s);
        }
    }
    big = __syncthreads_or(big);
    // V
    const int dp = (lane & 15) + 16 * (warp & 3), quarter = tile / 4, first = ((lane >> 4) + 2 * (warp >> 2)) * quarter;
    for (uint32_t bits = todo_of(s_todo, first, quarter); bits; bits &= bits - 1) {
        const int i = first + __ffs(bits) - 1, role = s_role[i];
        auto put = [&](int e, uint32_t w) { s_v[(i + e) * (HD / 2) + (dp ^ ((i + e) & 16))] = w; };
        if (role == 3) { put(0, 0u); continue; }
        const long long slot = s_slot[i];
        const int tl = (int)(slot & 63);
        const uint8_t *reg = chunk_of_page(a, layer, head, slot >> 6) + kv_region_bytes(a.k_type);
        if (VT == KV_T_F16) {
            const uint8_t *s0 = reg + v16_off(tl, 2 * dp), *s1 = reg + v16_off(tl, 2 * dp + 1);
            if (role == 2) {
                put(0, *reinterpret_cast<const uint16_t *>(s0) | ((uint32_t)*reinterpret_cast<const uint16_t *>(s1) << 16));
                continue;
            }
            const uint4 x = *reinterpret_cast<const uint4 *>(s0), y = *reinterpret_cast<const uint4 *>(s1);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; e++) put(e, __byte_perm(xw[e >> 1], yw[e >> 1], e & 1 ? 0x7632 : 0x5410));
        } else {
            const uint8_t *s0 = reg + v8_off(tl, 2 * dp), *s1 = reg + v8_off(tl, 2 * dp + 1);
            const uint32_t *sc = s_scale[i] + (dp >> 4);
            if (role == 2) {
                const uint32_t c = *s0 | ((uint32_t)*s1 << 8);
                put(0, VT == KV_T_FP8 ? e4m3x2_to_h2((uint16_t)c) : q8_pair(c, 0x4140, *sc, big));
                continue;
            }
            const uint4 x = *reinterpret_cast<const uint4 *>(s0), y = *reinterpret_cast<const uint4 *>(s1);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const uint32_t c = __byte_perm(xw[e >> 2], yw[e >> 2], e & 2 ? 0x7362 : 0x5140);   // both dims of two tokens
                if (VT == KV_T_FP8) {
                    put(e, e4m3x2_to_h2((uint16_t)c));
                    put(e + 1, e4m3x2_to_h2((uint16_t)(c >> 16)));
                } else {
                    put(e, q8_pair(c, 0x4140, sc[4 * e], big));
                    put(e + 1, q8_pair(c, 0x4342, sc[4 * e + 4], big));
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < AP_TILE / (2 * AP_WARPS); m++) {
        const int i = 2 * (warp + m * AP_WARPS) + (lane >> 4);
        if (i >= n) continue;
        const uint4 o = KT == KV_T_F16 ? kx[m] : decode8<KT>(make_uint2(kx[m].x, kx[m].y), ks[m]);
        __stcs(reinterpret_cast<uint4 *>(k + ((t0 + i) * a.n_kv + head) * HD + 8 * j), o);
    }
    __syncthreads();
#pragma unroll 4
    for (int i0 = 2 * warp; i0 < n; i0 += 2 * AP_WARPS) {
        const int i = i0 + (lane >> 4);
        if (i < n)
            __stcs(reinterpret_cast<uint4 *>(v + ((t0 + i) * a.n_kv + head) * HD + 8 * j),
                   *reinterpret_cast<const uint4 *>(s_v + i * (HD / 2) + ((4 * j) ^ (i & 16))));
    }
}

template <int KT>
static void read_of_key(unsigned grid, const KvPool &kv, int layer, int T, int tile, const int64_t *slots, uint16_t *k,
                        uint16_t *v, uint32_t *status, cudaStream_t stream) {
    switch (kv.v_type) {
        case KV_T_F16: chunk_read_kernel<KT, KV_T_F16><<<grid, AP_THREADS, 0, stream>>>(kv, layer, T, tile, slots, k, v, status); break;
        case KV_T_Q8: chunk_read_kernel<KT, KV_T_Q8><<<grid, AP_THREADS, 0, stream>>>(kv, layer, T, tile, slots, k, v, status); break;
        default: chunk_read_kernel<KT, KV_T_FP8><<<grid, AP_THREADS, 0, stream>>>(kv, layer, T, tile, slots, k, v, status); break;
    }
}
cudaError_t launch_chunk_read(const KvPool &kv, int layer, int T, const int64_t *slots, uint16_t *k, uint16_t *v,
                              uint32_t *status, cudaStream_t stream) {
    const int tile = value_tile(T, kv.n_kv);
    const long long ctas = ((long long)T + tile - 1) / tile * kv.n_kv;
    if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)ctas;
    switch (kv.k_type) {
        case KV_T_F16: read_of_key<KV_T_F16>(grid, kv, layer, T, tile, slots, k, v, status, stream); break;
        case KV_T_Q8: read_of_key<KV_T_Q8>(grid, kv, layer, T, tile, slots, k, v, status, stream); break;
        default: read_of_key<KV_T_FP8>(grid, kv, layer, T, tile, slots, k, v, status, stream); break;
    }
    return cudaGetLastError();
}

}  // namespace zdec
