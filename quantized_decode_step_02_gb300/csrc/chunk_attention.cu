// chunk_attention.cu -- attention of a chunk of new tokens over the paged cache.
#include "chunk.cuh"

namespace zdec {

size_t chunk_attention_workspace(int, int) { return 256; }

__device__ __forceinline__ float cached_k(const KvPool &kv, const uint8_t *reg, int t, int d) {
    if (kv.k_type == KV_T_F16) return __half2float(*reinterpret_cast<const __half *>(reg + k16_off(t, d)));
    const uint8_t c = reg[k8_off(t, d)];
    if (kv.k_type == KV_T_FP8) return __half2float(__ushort_as_half((uint16_t)(e4m3x2_to_h2(c) & 0xFFFFu)));
    return __half2float(*reinterpret_cast<const __half *>(reg + ks_off(t, d >> 5))) * (float)((int)c - 128);
}
__device__ __forceinline__ float cached_v(const KvPool &kv, const uint8_t *reg, int t, int d) {
    if (kv.v_type == KV_T_F16) return __half2float(*reinterpret_cast<const __half *>(reg + v16_off(t, d)));
    const uint8_t c = reg[v8_off(t, d)];
    if (kv.v_type == KV_T_FP8) return __half2float(__ushort_as_half((uint16_t)(e4m3x2_to_h2(c) & 0xFFFFu)));
    return __half2float(*reinterpret_cast<const __half *>(reg + vs_off(t, d >> 5))) * (float)((int)c - 128);
}

// One warp per (token, query head), lane l: dims l + 32 i; one pass over the
// keys with the running maximum and sum.
__global__ void chunk_attention_kernel(const ChunkAttnParams p) {
    const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (w >= (long long)p.T * p.nq) return;
    const int t = (int)(w / p.nq), h = (int)(w % p.nq);
    if (t >= p.cu[p.R]) return;
    int a = 0, b = p.R;   // the last request that starts at or before t
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (p.cu[m] <= t) a = m;
        else b = m;
    }
    const int n = p.cu[a + 1] - p.cu[a], i = t - p.cu[a];
    const long long cap = (long long)p.kv.max_pages * 64;
    const int kv_len = (int)min(cap, (long long)max(0, p.kv_len[a]));
    long long hi = kv_len, lo = 0;
    if (p.causal) {
        const long long pos = (long long)p.kv_len[a] - n + i;
        hi = min(hi, pos + 1);
        if (p.window) lo = max(0LL, pos + 1 - p.window);
    }
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.0f;
    for (int e = 0; e < 4; e++) {
        const uint16_t x = p.q[(long long)t * p.q_ld + (long long)h * HD + lane + 32 * e];
        q[e] = (p.io_type == ZDEC_F16 ? __half2float(__ushort_as_half(x)) : __uint_as_float((uint32_t)x << 16)) * p.scale_log2;
    }
    for (long long j = lo; j < hi; j++) {
        const int page = p.kv.table[(size_t)a * p.kv.max_pages + (j >> 6)];
        if (!kv_page_ok(p.kv, page)) {
            if (p.status && lane == 0) atomicOr(p.status, (uint32_t)ZDEC_CHUNK_NO_PAGE);
            j |= 63;
            continue;
        }
        const uint8_t *kr = p.kv.base + (size_t)page * p.kv.page_bytes + kv_chunk_off(p.kv, p.layer, h / p.G);
        const uint8_t *vr = kr + kv_region_bytes(p.kv.k_type);
        float s = 0.0f;
        for (int e = 0; e < 4; e++) s = fmaf(q[e], cached_k(p.kv, kr, (int)(j & 63), lane + 32 * e), s);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
        const float mn = fmaxf(m, s), f = exp2f(m - mn), pr = exp2f(s - mn);
        for (int e = 0; e < 4; e++) o[e] = o[e] * f + pr * cached_v(p.kv, vr, (int)(j & 63), lane + 32 * e);
        l = l * f + pr;
        m = mn;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    for (int e = 0; e < 4; e++) {
        const float y = o[e] * inv;
        uint32_t bf;
        asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(bf) : "f"(y));
        p.o[(long long)t * p.o_ld + (long long)h * HD + lane + 32 * e] =
            p.io_type == ZDEC_F16 ? __half_as_ushort(__float2half_rn(y)) : (uint16_t)bf;
    }
}

cudaError_t launch_chunk_attention(const ChunkAttnParams &p, cudaStream_t stream) {
    const long long blocks = ((long long)p.T * p.nq * 32 + 255) / 256;
    chunk_attention_kernel<<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace zdec
