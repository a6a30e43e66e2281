// spec_attention.cu -- attention of the nodes of draft trees over the paged
// 8-bit cache and each other.
#include <math.h>

#include "cache_device.cuh"
#include "internal.h"

using namespace svc;

namespace {

struct Att {
    int B, N, Hq, Hkv, G, D, page;
    sv_host::Rows q, k, v;
    spec_kv_cache c;
    const uint32_t* anc;          // nullable: chains
    float scale;                  // scale * log2(e)
    char* out;
    float* lse;
    unsigned* status;
};

__device__ __forceinline__ float e4m3_f32(uint8_t v) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"((uint32_t)v));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

// One warp per row (b, n, query head): each lane holds D / 32 elements of q and
// of the sum, every key is one dot product over the warp, with the running
// maximum and sum of the softmax.
template <int D>
__global__ void __launch_bounds__(128) k_attention_rows(const Att P) {
    constexpr int E = D / 32;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (int64_t)P.B * P.N * P.Hq) return;
    const int h = row % P.Hq, n = row / P.Hq % P.N, b = row / P.Hq / P.N, hk = h / P.G;
    const int page = P.page;
    const int len = P.c.lengths[b];
    const int slot = P.c.slots ? P.c.slots[b] : b;
    const int64_t most = (int64_t)P.c.max_pages * page + page - 1;
    bool bad = len >= 0 && (len > most || len >= SPEC_MAX_CACHE_LEN || slot < 0 || slot >= P.c.num_slots);
    float q[E], acc[E] = {}, m = -INFINITY, l = 0.f;
    const __nv_bfloat16* qp = reinterpret_cast<const __nv_bfloat16*>(P.q.p + b * P.q.b + n * P.q.n + h * P.q.h);
#pragma unroll
    for (int i = 0; i < E; ++i) q[i] = __bfloat162float(qp[lane * E + i]);
    auto key = [&](const float (&k)[E], const float (&v)[E]) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
        s *= P.scale;
        const float m2 = fmaxf(m, s);
        const float old = m2 == -INFINITY ? 1.f : exp2f(m - m2), p = m2 == -INFINITY ? 0.f : exp2f(s - m2);
        l = l * old + p;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = acc[i] * old + p * v[i];
        m = s != s ? s : m2;
    };
    if (!bad && len >= 0) {
        const int full = len / page;
        for (int j = 0; j < full && !bad; ++j) {
            const int id = P.c.page_table[b * P.c.page_table_stride + j];
            if (id < 0 || id >= P.c.num_pages) {
                bad = true;
                break;
            }
            const int64_t ph = (int64_t)id * P.Hkv + hk;
            const uint8_t* kp = static_cast<const uint8_t*>(P.c.k_pages) + ph * page * D;
            const uint8_t* vp = static_cast<const uint8_t*>(P.c.v_pages) + ph * page * D;
            const float ks = P.c.k_scale[ph], vs = P.c.v_scale[ph];
            for (int t = 0; t < page; ++t) {
                float k[E], v[E];
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    k[i] = e4m3_f32(kp[t * D + lane * E + i]) * ks;
                    v[i] = e4m3_f32(vp[t * D + lane * E + i]) * vs;
                }
                key(k, v);
            }
        }
        for (int t = full * page; t < len; ++t) {
            const int64_t at = (((int64_t)slot * P.Hkv + hk) * 2 * page + t % (2 * page)) * D;
            const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(P.c.k_open) + at;
            const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(P.c.v_open) + at;
            float k[E], v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                k[i] = __bfloat162float(kp[lane * E + i]);
                v[i] = __bfloat162float(vp[lane * E + i]);
            }
            key(k, v);
        }
        const int W = (P.N + 31) / 32;
        for (int t = 0; t < P.N; ++t) {
            const bool sees = P.anc ? (P.anc[((int64_t)b * P.N + n) * W + t / 32] >> (t & 31)) & 1 : t <= n;
            if (!sees) continue;
            const __nv_bfloat16* kp = reinterpret_cast<const __nv_bfloat16*>(P.k.p + b * P.k.b + t * P.k.n + hk * P.k.h);
            const __nv_bfloat16* vp = reinterpret_cast<const __nv_bfloat16*>(P.v.p + b * P.v.b + t * P.v.n + hk * P.v.h);
            float k[E], v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                k[i] = __bfloat162float(kp[lane * E + i]);
                v[i] = __bfloat162float(vp[lane * E + i]);
            }
            key(k, v);
        }
    }
    const float nan = __int_as_float(0x7fffffff);
    if (bad && lane == 0) atomicOr(P.status, 1u << SPEC_ERR_DEVICE_INPUT);
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(P.out) + row * D;
#pragma unroll
    for (int i = 0; i < E; ++i) o[lane * E + i] = __float2bfloat16(bad ? nan : acc[i] * inv);
    if (P.lse && lane == 0)
        P.lse[row] = bad ? nan : l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace

using sv_host::fail;

extern "C" {

size_t spec_cache_workspace_bytes(int B, int N, int q_heads, int head_dim) {
    if (B < 0 || B > sv_host::CACHE_MAX_B || N < 1 || N > SPEC_MAX_NODES || q_heads < 1 || q_heads > SPEC_MAX_HEADS ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    return sv_host::CACHE_WS_PARTIAL;
}

spec_status spec_tree_attention(int B, int N, int q_heads, const spec_kv_cache* cache,
                                const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                                const void* v, const int64_t* v_strides,
                                const int32_t* ancestors, float scale, void* out, float* lse,
                                void* workspace, size_t workspace_bytes, void* stream) {
    sv_host::Range range("spec_tree_attention");
    if (B < 0 || B > sv_host::CACHE_MAX_B)
        return fail(SPEC_ERR_INVALID_ARG, "B %d outside [0, %d]", B, sv_host::CACHE_MAX_B);
    if (N < 1 || N > SPEC_MAX_NODES) return fail(SPEC_ERR_INVALID_ARG, "N %d outside [1, %d]", N, SPEC_MAX_NODES);
    if (spec_status s = sv_host::check_cache(cache, B)) return s;
    if (q_heads < 1 || q_heads > SPEC_MAX_HEADS || q_heads % cache->kv_heads != 0)
        return fail(SPEC_ERR_INVALID_ARG, "q_heads %d is not a multiple of kv_heads %d up to %d", q_heads,
                    cache->kv_heads, SPEC_MAX_HEADS);
    if (!(scale > 0.f) || scale > 3.402823466e38f)
        return fail(SPEC_ERR_INVALID_ARG, "scale is not a positive finite value");
    if (B == 0) return SPEC_OK;
    Att P{};
    const int D = cache->head_dim;
    if (spec_status s = sv_host::make_rows("q", q, q_strides, B, N, q_heads, 2, &P.q)) return s;
    if (spec_status s = sv_host::make_rows("k", k, k_strides, B, N, cache->kv_heads, 2, &P.k)) return s;
    if (spec_status s = sv_host::make_rows("v", v, v_strides, B, N, cache->kv_heads, 2, &P.v)) return s;
    if (!out) return fail(SPEC_ERR_INVALID_ARG, "out is NULL");
    if (((uintptr_t)out & 15u) != 0) return fail(SPEC_ERR_INVALID_ARG, "out not 16-byte aligned");
    if (spec_status s = sv_host::check_cache_ws(workspace, workspace_bytes, spec_cache_workspace_bytes(B, N, q_heads, D)))
        return s;
    P.B = B; P.N = N; P.Hq = q_heads; P.Hkv = cache->kv_heads; P.G = q_heads / cache->kv_heads; P.D = D;
    P.page = cache->page_size;
    P.c = *cache;
    P.anc = reinterpret_cast<const uint32_t*>(ancestors);
    P.scale = (float)((double)scale * 1.4426950408889634073599);
    P.out = static_cast<char*>(out);
    P.lse = lse;
    P.status = static_cast<unsigned*>(workspace);
    const int64_t rows = (int64_t)B * N * q_heads;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (D == 64) k_attention_rows<64><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(P);
    else k_attention_rows<128><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(P);
    return sv_host::launched("k_attention_rows");
}

}  // extern "C"
