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
// always one of the new tokens.
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
template <int T>
struct InType;
template <>
struct InType<ZDEC_F32> {
    static __device__ __forceinline__ float2 load2(const void *p, long long i) {
        return __ldg(reinterpret_cast<const float2 *>(static_cast<const float *>(p) + i));
    }
    static __device__ __forceinline__ float4 load4(const void *p, long long i) {
        return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
    }
};
template <>
struct InType<ZDEC_F16> {
    static __device__ __forceinline__ float2 load2(const void *p, long long i) {
        return __half22float2(u32_as_h2(__ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i))));
    }
    static __device__ __forceinline__ float4 load4(const void *p, long long i) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i));
        const float2 a = __half22float2(u32_as_h2(w.x)), b = __half22float2(u32_as_h2(w.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
};
__device__ __forceinline__ float2 bf2_to_f2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
struct InType<ZDEC_BF16> {
    static __device__ __forceinline__ float2 load2(const void *p, long long i) {
        return bf2_to_f2(__ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i)));
    }
    static __device__ __forceinline__ float4 load4(const void *p, long long i) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i));
        const float2 a = bf2_to_f2(w.x), b = bf2_to_f2(w.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
};
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {   // nearest even, low half x
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) { return h2_as_u32(__floats2half2_rn(x, y)); }

// Two fp16 values -> two stored bytes (low first): e4m3, or Q8_0 codes + 128
// of a block with fp32 scale d (0 for an all-zero block).
__device__ __forceinline__ uint16_t fp8_pair(uint32_t h2) {
    uint16_t out;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(out) : "r"(h2));
    return out;
}
__device__ __forceinline__ uint32_t q8_code(float x, float d) {
    if (d == 0.0f) return 128u;
    const int q = max(-127, min(127, __float2int_rn(__fdiv_rn(x, d))));
    return (uint32_t)(q + 128) & 0xFFu;
}
// A block's scale from its amax: fp32 IEEE division (0 for an all-zero block).
__device__ __forceinline__ float q8_scale(float amax) { return amax == 0.0f ? 0.0f : __fdiv_rn(amax, 127.0f); }

constexpr int AP_THREADS = 256, AP_WARPS = AP_THREADS / 32, AP_TILE = 64;   // AP_TILE: tokens of a value-head CTA

// Rotation of the query and key heads: a warp takes tokens and a share of the
// heads; lane l holds the pairs 2l and 2l + 1, whose angles it computes once
// per token.
template <int IN, int KT>
__device__ __forceinline__ void append_qk(const ChunkAppendParams &p, int tile, int split, const unsigned long long *s_turn,
                                          const uint8_t *s_axis) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = p.nq + p.kv.n_kv;
    const int h0 = (int)((long long)heads * split / p.splits), h1 = (int)((long long)heads * (split + 1) / p.splits);
    const unsigned long long turn0 = s_turn[2 * lane], turn1 = s_turn[2 * lane + 1];
    const int ax0 = s_axis[2 * lane], ax1 = s_axis[2 * lane + 1];
    const int tile_tok = AP_WARPS * p.tok_warp;
    for (int i = 0; i < p.tok_warp; i++) {
        const long long t = (long long)tile * tile_tok + i * AP_WARPS + warp;
        if (t >= p.T) break;
        float s0, c0, s1, c1;
        {
            const long long a = __ldg(p.positions + (size_t)ax0 * p.T + t), b = __ldg(p.positions + (size_t)ax1 * p.T + t);
            // position * turns mod 1 in 0.64 fixed point; the signed high word is the angle in half turns / 2^31
            const int fa = (int)(((unsigned long long)a * turn0) >> 32), fb = (int)(((unsigned long long)b * turn1) >> 32);
            sincospif((float)fa * 4.656612873077393e-10f, &s0, &c0);
            sincospif((float)fb * 4.656612873077393e-10f, &s1, &c1);
        }
        const long long slot = h1 > p.nq ? checked_slot(p.kv, __ldg(p.slots + t), p.status) : -1;
        const long long row = t * p.ld;
#pragma unroll 4
        for (int h = h0; h < h1; h++) {
            const float2 a = InType<IN>::load2(p.qkv, row + (long long)h * HD + 2 * lane);
            const float2 b = InType<IN>::load2(p.qkv, row + (long long)h * HD + 64 + 2 * lane);
            const float x0 = a.x * c0 - b.x * s0, x1 = a.y * c1 - b.y * s1;
            const float y0 = b.x * c0 + a.x * s0, y1 = b.y * c1 + a.y * s1;
            if (h < p.nq) {
                uint32_t *q = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.q_out) + t * p.q_ld + (long long)h * HD + 2 * lane);
                q[0] = p.q_type == ZDEC_F16 ? pack_f16(x0, x1) : pack_bf16(x0, x1);
                q[32] = p.q_type == ZDEC_F16 ? pack_f16(y0, y1) : pack_bf16(y0, y1);
                continue;
            }
            if (slot < 0) continue;   // the whole warp: one token
            uint8_t *reg = chunk_of_page(p.kv, p.layer, h - p.nq, slot >> 6);
            const int tl = (int)(slot & 63);
            const uint32_t hx = pack_f16(x0, x1), hy = pack_f16(y0, y1);
            if (KT == KV_T_F16) {
                *reinterpret_cast<uint32_t *>(reg + k16_off(tl, 2 * lane)) = hx;
                *reinterpret_cast<uint32_t *>(reg + k16_off(tl, 64 + 2 * lane)) = hy;
            } else if (KT == KV_T_FP8) {
                *reinterpret_cast<uint16_t *>(reg + k8_off(tl, 2 * lane)) = fp8_pair(hx);
                *reinterpret_cast<uint16_t *>(reg + k8_off(tl, 64 + 2 * lane)) = fp8_pair(hy);
            } else {
                // blocks of 32 dims: lanes 0-15 hold blocks 0 and 2, lanes 16-31 blocks 1 and 3
                const float2 fx = __half22float2(u32_as_h2(hx)), fy = __half22float2(u32_as_h2(hy));
                float mx = fmaxf(fabsf(fx.x), fabsf(fx.y)), my = fmaxf(fabsf(fy.x), fabsf(fy.y));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) {
                    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
                    my = fmaxf(my, __shfl_xor_sync(FULL, my, o));
                }
                const float dx = q8_scale(mx), dy = q8_scale(my);
                *reinterpret_cast<uint16_t *>(reg + k8_off(tl, 2 * lane)) = (uint16_t)(q8_code(fx.x, dx) | (q8_code(fx.y, dx) << 8));
                *reinterpret_cast<uint16_t *>(reg + k8_off(tl, 64 + 2 * lane)) = (uint16_t)(q8_code(fy.x, dy) | (q8_code(fy.y, dy) << 8));
                if ((lane & 15) == 0) {
                    *reinterpret_cast<uint16_t *>(reg + ks_off(tl, lane >> 4)) = __half_as_ushort(__float2half_rn(dx));
                    *reinterpret_cast<uint16_t *>(reg + ks_off(tl, 2 + (lane >> 4))) = __half_as_ushort(__float2half_rn(dy));
                }
            }
        }
    }
}

// One value head of up to AP_TILE tokens: encoded rows meet in shared memory
// and leave transposed, 16 bytes (SEG tokens of one dim) at a time where SEG
// tokens of the tile fill one 16-byte segment of the page, else element by
// element.
template <int IN, int VT>
__device__ __forceinline__ void append_v(const ChunkAppendParams &p, int tile, int head, uint8_t *smem, long long *s_slot) {
    constexpr int ES = VT == KV_T_F16 ? 2 : 1, SEG = 16 / ES;
    constexpr int PITCH = HD * ES + 4;   // bytes of a row: 4 more, so that the rows of a column fall in different banks
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t0 = (long long)tile * AP_TILE;
    const int n = (int)min((long long)AP_TILE, p.T - t0);
    if ((int)threadIdx.x < AP_TILE)
        s_slot[threadIdx.x] = (int)threadIdx.x < n ? checked_slot(p.kv, __ldg(p.slots + t0 + threadIdx.x), p.status) : -1;
    __syncthreads();
    const long long col = (long long)(p.nq + p.kv.n_kv + head) * HD;
#pragma unroll 4
    for (int i = warp; i < n; i += AP_WARPS) {
        const float4 x = InType<IN>::load4(p.qkv, (t0 + i) * p.ld + col + 4 * lane);
        const uint32_t h0 = pack_f16(x.x, x.y), h1 = pack_f16(x.z, x.w);
        uint8_t *row = smem + i * PITCH;
        if (VT == KV_T_F16) {
            *reinterpret_cast<uint32_t *>(row + 8 * lane) = h0;
            *reinterpret_cast<uint32_t *>(row + 8 * lane + 4) = h1;
        } else if (VT == KV_T_FP8) {
            *reinterpret_cast<uint32_t *>(row + 4 * lane) = (uint32_t)fp8_pair(h0) | ((uint32_t)fp8_pair(h1) << 16);
        } else {
            const float2 a = __half22float2(u32_as_h2(h0)), b = __half22float2(u32_as_h2(h1));
            float m = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y)));
            m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));   // a block of 32 dims: 8 lanes
            m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
            m = fmaxf(m, __shfl_xor_sync(FULL, m, 4));
            const float d = q8_scale(m);
            *reinterpret_cast<uint32_t *>(row + 4 * lane) =
                q8_code(a.x, d) | (q8_code(a.y, d) << 8) | (q8_code(b.x, d) << 16) | (q8_code(b.y, d) << 24);
            const long long slot = s_slot[i];
            if ((lane & 7) == 0 && slot >= 0) {
                uint8_t *reg = chunk_of_page(p.kv, p.layer, head, slot >> 6) + kv_region_bytes(p.kv.k_type);
                *reinterpret_cast<uint16_t *>(reg + vs_off((int)(slot & 63), lane >> 3)) = __half_as_ushort(__float2half_rn(d));
            }
        }
    }
    __syncthreads();
    // thread: dim d, tokens i = i0, i0 + 2, ...: a token that opens a whole
    // segment stores it, one inside a whole segment does nothing
    const int d = threadIdx.x & (HD - 1);
    for (int i = threadIdx.x >> 7; i < n; i += AP_THREADS / HD) {
        const long long slot = s_slot[i];
        if (slot < 0) continue;
        const int in = (int)(slot & (SEG - 1)), a = i - in;   // a: where the segment's first token would be
        bool whole = a >= 0 && a + SEG <= n;
        if (whole)
            for (int e = 0; e < SEG; e++) whole = whole && s_slot[a + e] == slot - in + e;
        if (whole && in != 0) continue;
        uint8_t *reg = chunk_of_page(p.kv, p.layer, head, slot >> 6) + kv_region_bytes(p.kv.k_type);
        const int tl = (int)(slot & 63);
        if (VT == KV_T_F16) {
            uint8_t *dst = reg + v16_off(tl, d);
            const uint16_t *src = reinterpret_cast<const uint16_t *>(smem + i * PITCH) + d;
            if (whole) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    w[e] = (uint32_t)src[(2 * e) * (PITCH / 2)] | ((uint32_t)src[(2 * e + 1) * (PITCH / 2)] << 16);
                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                *reinterpret_cast<uint16_t *>(dst) = src[0];
            }
        } else {
            uint8_t *dst = reg + v8_off(tl, d);
            const uint8_t *src = smem + i * PITCH + d;
            if (whole) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    w[e] = (uint32_t)src[(4 * e) * PITCH] | ((uint32_t)src[(4 * e + 1) * PITCH] << 8) |
                           ((uint32_t)src[(4 * e + 2) * PITCH] << 16) | ((uint32_t)src[(4 * e + 3) * PITCH] << 24);
                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                *dst = src[0];
            }
        }
    }
}

// grid (token tiles, splits + value heads): y < splits rotate, the others move values.
template <int IN>
__global__ __launch_bounds__(AP_THREADS) void chunk_append_kernel(const __grid_constant__ ChunkAppendParams p) {
    __shared__ unsigned long long s_turn[64];
    __shared__ uint8_t s_axis[64];
    __shared__ long long s_slot[AP_TILE];
    __shared__ __align__(16) uint8_t s_v[AP_TILE * (HD * 2 + 4)];
    if ((int)blockIdx.y < p.splits) {
        if (threadIdx.x < 64) {
            s_turn[threadIdx.x] = p.rope.turn[threadIdx.x];
            s_axis[threadIdx.x] = p.rope.axis[threadIdx.x];
        }
        __syncthreads();
        for (long long tile = blockIdx.x; tile * AP_WARPS * p.tok_warp < p.T; tile += gridDim.x) {
            switch (p.kv.k_type) {
                case KV_T_F16: append_qk<IN, KV_T_F16>(p, (int)tile, blockIdx.y, s_turn, s_axis); break;
                case KV_T_Q8: append_qk<IN, KV_T_Q8>(p, (int)tile, blockIdx.y, s_turn, s_axis); break;
                default: append_qk<IN, KV_T_FP8>(p, (int)tile, blockIdx.y, s_turn, s_axis); break;
            }
        }
    } else {
        for (long long tile = blockIdx.x; tile * AP_TILE < p.T; tile += gridDim.x) {
            for (int head = blockIdx.y - p.splits; head < p.kv.n_kv; head += gridDim.y - p.splits) {
                switch (p.kv.v_type) {
                    case KV_T_F16: append_v<IN, KV_T_F16>(p, (int)tile, head, s_v, s_slot); break;
                    case KV_T_Q8: append_v<IN, KV_T_Q8>(p, (int)tile, head, s_v, s_slot); break;
                    default: append_v<IN, KV_T_FP8>(p, (int)tile, head, s_v, s_slot); break;
                }
                __syncthreads();
            }
        }
    }
}

cudaError_t launch_chunk_append(ChunkAppendParams p, cudaStream_t stream) {
    const int heads = p.nq + p.kv.n_kv;
    p.tok_warp = AP_TILE / AP_WARPS;
    p.splits = std::max(1, std::min(heads, 8));
    const long long tiles = ((long long)p.T + AP_TILE - 1) / AP_TILE;
    const dim3 grid((unsigned)std::min(tiles, 1LL << 20), (unsigned)(p.splits + std::min(p.kv.n_kv, 4096)));
    switch (p.in_type) {
        case ZDEC_F32: chunk_append_kernel<ZDEC_F32><<<grid, AP_THREADS, 0, stream>>>(p); break;
        case ZDEC_F16: chunk_append_kernel<ZDEC_F16><<<grid, AP_THREADS, 0, stream>>>(p); break;
        default: chunk_append_kernel<ZDEC_BF16><<<grid, AP_THREADS, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

// ------------------------------------------------------------------ read ---
// A stored Q8_0 code times its scale, exact in fp32, at most fp16's largest
// value (127 x a scale of 516 lies past it).
__device__ __forceinline__ float q8_value(float scale, uint32_t code) {
    const float x = scale * (float)((int)code - 128);
    return x > 65504.0f ? 65504.0f : (x < -65504.0f ? -65504.0f : x);
}
// One warp per (token, kv head), lane l: dims 4l .. 4l + 3 of K and V.
__global__ void chunk_read_kernel(const KvPool a, int layer, int T, const int64_t *__restrict__ slots,
                                  uint16_t *__restrict__ k, uint16_t *__restrict__ v, uint32_t *status) {
    const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (w >= (long long)T * a.n_kv) return;
    const long long t = w / a.n_kv;
    const int g = (int)(w % a.n_kv);
    const long long slot = checked_slot(a, slots[t], status);
    uint2 ko = make_uint2(0u, 0u), vo = ko;
    if (slot >= 0) {
        const uint8_t *kr = chunk_of_page(a, layer, g, slot >> 6), *vr = kr + kv_region_bytes(a.k_type);
        const int tl = (int)(slot & 63), d = 4 * lane;
        if (a.k_type == KV_T_F16) {
            ko = *reinterpret_cast<const uint2 *>(kr + k16_off(tl, d));
        } else {
            const uint32_t c = *reinterpret_cast<const uint32_t *>(kr + k8_off(tl, d));
            if (a.k_type == KV_T_FP8) {
                ko = make_uint2(e4m3x2_to_h2((uint16_t)c), e4m3x2_to_h2((uint16_t)(c >> 16)));
            } else {
                const float s = __half2float(*reinterpret_cast<const __half *>(kr + ks_off(tl, lane >> 3)));
                float f[4];
                for (int e = 0; e < 4; e++) f[e] = q8_value(s, (c >> (8 * e)) & 255u);
                ko = make_uint2(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]));
            }
        }
        uint16_t e4[4];
        float s = 1.0f;
        if (a.v_type == KV_T_Q8) s = __half2float(*reinterpret_cast<const __half *>(vr + vs_off(tl, lane >> 3)));
        for (int e = 0; e < 4; e++) {
            if (a.v_type == KV_T_F16) e4[e] = *reinterpret_cast<const uint16_t *>(vr + v16_off(tl, d + e));
            else {
                const uint8_t c = vr[v8_off(tl, d + e)];
                e4[e] = a.v_type == KV_T_FP8 ? (uint16_t)(e4m3x2_to_h2(c) & 0xFFFFu)
                                             : __half_as_ushort(__float2half_rn(q8_value(s, c)));
            }
        }
        vo = make_uint2((uint32_t)e4[0] | ((uint32_t)e4[1] << 16), (uint32_t)e4[2] | ((uint32_t)e4[3] << 16));
    }
    *reinterpret_cast<uint2 *>(k + w * HD + 4 * lane) = ko;
    *reinterpret_cast<uint2 *>(v + w * HD + 4 * lane) = vo;
}

cudaError_t launch_chunk_read(const KvPool &kv, int layer, int T, const int64_t *slots, uint16_t *k, uint16_t *v,
                              uint32_t *status, cudaStream_t stream) {
    const long long warps = (long long)T * kv.n_kv;
    const long long blocks = (warps * 32 + 255) / 256;
    if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    chunk_read_kernel<<<(unsigned)blocks, 256, 0, stream>>>(kv, layer, T, slots, k, v, status);
    return cudaGetLastError();
}

}  // namespace zdec
