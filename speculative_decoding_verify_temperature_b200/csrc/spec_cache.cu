// spec_cache.cu -- the cache calls around a verify round, except the attention
// itself: the plan of the draft trees, the norm and rotation of queries and
// keys, the append of accepted rows to the paged 8-bit cache.
#include <stdio.h>

#include "cache_device.cuh"
#include "internal.h"

using namespace svc;

namespace {

// ----------------------------------------------------------------------------- plan

// One CTA per sequence, thread n = node n.  Parents go to shared memory; each
// node climbs to the root, which takes its depth in steps of one shared load.
// Node ids fall on the way up, so the word of the mask being filled changes at
// most W times and stays in a register.  Bound by latency: the climb and the launch
// (256 trees of 256 nodes, 2.6 MB written: 13 us a call, as one node of one tree; the host's part of the call).
constexpr int PLAN_MAXW = SPEC_MAX_NODES / 32;

__global__ void __launch_bounds__(SPEC_MAX_NODES) k_tree_plan(int N, int max_depth, const int32_t* __restrict__ parents,
                                                              const int32_t* __restrict__ lengths, int32_t* out_pos,
                                                              uint32_t* out_anc, unsigned* status) {
    __shared__ int par[SPEC_MAX_NODES];
    __shared__ uint32_t anc[SPEC_MAX_NODES * PLAN_MAXW];
    const int b = blockIdx.x, n = threadIdx.x, W = (N + 31) / 32;
    const int len = lengths[b];
    int p = -1;
    bool bad = len >= SPEC_MAX_CACHE_LEN;
    if (n < N && len >= 0) {              // the parents of a row without a sequence are not looked at
        p = parents ? parents[(int64_t)b * N + n] : n - 1;
        bad |= n == 0 ? p != -1 : (p < 0 || p >= n);
        par[n] = p;
        for (int w = 0; w < W; ++w) anc[n * W + w] = 0;
    }
    bad = __syncthreads_or(bad);
    int depth = 0;
    if (!bad && len >= 0 && n < N) {
        int cur = n;
        uint32_t word = 0;
        while (true) {
            word |= 1u << (cur & 31);
            const int up = par[cur];
            if (up < 0 || (up >> 5) != (cur >> 5)) {
                anc[n * W + (cur >> 5)] = word;
                word = 0;
            }
            if (up < 0) break;
            cur = up;
            ++depth;
        }
    }
    // chains (no parents given) may be deeper than a tree's limit
    bad = __syncthreads_or(bad || (parents && depth > max_depth));
    const bool off = bad || len < 0;
    if (bad && n == 0) atomicOr(status, 1u << SPEC_ERR_DEVICE_INPUT);
    if (n < N) out_pos[(int64_t)b * N + n] = off ? -1 : len + depth;
    uint32_t* dst = out_anc + (int64_t)b * N * W;
    for (int i = n; i < N * W; i += blockDim.x) dst[i] = off ? 0u : anc[i];
}

// ----------------------------------------------------------------------------- norm + rotation

struct NormRope {
    int B, N, Hq, Hk, D, rot, interleaved, GW;
    sv_host::Rows q, k, qo, ko;
    const int32_t* pos;
    const float* inv_freq;
    const char *qw, *kw;
    int w_f32;
    float eps;
};

constexpr int NR_BT = 128;
constexpr int NR_U = 3;                 // head rows in flight per group of lanes

__device__ __forceinline__ float weight_at(const char* w, int f32, int e) {
    return f32 ? __ldg(reinterpret_cast<const float*>(w) + e)
               : __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(w) + e) << 16);
}

// A CTA holds one token and some of its heads: a group of GW lanes takes a head
// row, eight elements per lane, both elements of a rotated pair in the same one, so
// that the only traffic between lanes is the sum of squares.  The angles of a
// token are the same for all of its heads: each is formed once per CTA, in f64,
// while the first rows are on their way.  Each element is read and written once: 32 x 64 tokens of 72 bf16 heads of 128, 75 MB,
// take 24.5 us, 3.1 TB/s (0.47 of the copy rate; what was written before stays in L2, DRAM is 20% busy).  Bound by
// instructions: 59% of the issue slots, about 23 per element and lane with the angles.
template <int DT>
__global__ void __launch_bounds__(NR_BT) k_norm_rope(const NormRope P) {
    __shared__ __align__(16) float cs[2][128], wt[2][256];
    constexpr int ESZ = Quad<DT>::ESZ;
    const int tok = blockIdx.x, b = tok / P.N, n = tok - b * P.N;
    const int GW = P.GW, l = threadIdx.x & (GW - 1);
    const int groups = NR_BT / GW, grp = threadIdx.x / GW;
    const int heads = P.Hq + P.Hk;
    const int per = (heads + gridDim.y - 1) / gridDim.y;
    const int h0 = blockIdx.y * per, h1 = min(heads, h0 + per);
    const bool on = 8 * l < P.D;
    const Quads at(l, P.rot, P.interleaved);
    const char* q = P.q.p + b * P.q.b + n * P.q.n;
    const char* k = P.k.p + b * P.k.b + n * P.k.n;
    char* qo = P.qo.p + b * P.qo.b + n * P.qo.n;
    char* ko = P.ko.p + b * P.ko.b + n * P.ko.n;
    const int o0 = at.q0 * 4 * ESZ, o1 = at.q1 * 4 * ESZ;
    const int pos = P.pos[tok];
    const float inv_d = 1.f / (float)P.D;
    float4 c, s;
    for (int base = h0; base < h1; base += groups * NR_U) {
        Quad<DT> r[NR_U][2];
#pragma unroll
        for (int u = 0; u < NR_U; ++u) {
            const int h = base + u * groups + grp;
            r[u][0].zero();
            r[u][1].zero();
            if (h < h1 && on && pos >= 0) {
                const char* p = h < P.Hq ? q + h * P.q.h : k + (h - P.Hq) * P.k.h;
                r[u][0].load(p + o0);
                r[u][1].load(p + o1);
            }
        }
        if (base == h0) {
            if (pos >= 0)
                for (int j = threadIdx.x; j < P.rot / 2; j += NR_BT) {
                    const float2 v = cos_sin(pos, P.inv_freq[j]);
                    cs[0][j] = v.x;
                    cs[1][j] = v.y;
                }
            if (P.qw || P.kw)
                for (int e = threadIdx.x; e < P.D; e += NR_BT) {
                    if (P.qw) wt[0][e] = weight_at(P.qw, P.w_f32, e);
                    if (P.kw) wt[1][e] = weight_at(P.kw, P.w_f32, e);
                }
            __syncthreads();
            if (at.turns) {
                c = *reinterpret_cast<const float4*>(&cs[0][4 * l]);
                s = *reinterpret_cast<const float4*>(&cs[1][4 * l]);
            }
        }
#pragma unroll
        for (int u = 0; u < NR_U; ++u) {
            if (base + u * groups >= h1) break;           // the same for the whole CTA
            const int h = base + u * groups + grp;
            float x[8];
            r[u][0].get(x);
            r[u][1].get(x + 4);
            if (P.qw || P.kw) {                           // a warp may hold query and key rows: all lanes reduce
                const float rs = row_rms(x, GW, inv_d, P.eps);
                if ((h < P.Hq ? P.qw : P.kw) != nullptr && on) {
                    const float* w = wt[h < P.Hq ? 0 : 1];
                    const float4 w0 = *reinterpret_cast<const float4*>(w + 4 * at.q0), w1 = *reinterpret_cast<const float4*>(w + 4 * at.q1);
                    x[0] = x[0] * rs * w0.x; x[1] = x[1] * rs * w0.y; x[2] = x[2] * rs * w0.z; x[3] = x[3] * rs * w0.w;
                    x[4] = x[4] * rs * w1.x; x[5] = x[5] * rs * w1.y; x[6] = x[6] * rs * w1.z; x[7] = x[7] * rs * w1.w;
                }
            }
            if (at.turns) row_rotate(x, c, s, P.interleaved);
            if (h < h1 && on) {
                if (pos < 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = 0.f;
                }
                char* p = h < P.Hq ? qo + h * P.qo.h : ko + (h - P.Hq) * P.ko.h;
                r[u][0].set(x);
                r[u][1].set(x + 4);
                r[u][0].store(p + o0);
                r[u][1].store(p + o1);
            }
        }
    }
}

// ----------------------------------------------------------------------------- append

struct Append {
    int B, T, W, Hkv, D, page, rot, interleaved, w_f32, GW;
    int heads_per_cta;
    sv_host::Rows k, v;
    spec_kv_cache c;
    const int32_t *num_accepted, *index;
    const float* inv_freq;
    const char* kw;
    float eps;
    int32_t* out_lengths;
    unsigned *status, *cnt;
};

constexpr int AP_BT = 256;

// Exponent bits of a block's scale, from the bits of its largest (bf16) magnitude: the least power of two s, 2^-126 or
// more, with amax / s <= 448 = 1.75 * 2^8; 1 for a block of zeros.
__device__ __forceinline__ uint32_t block_scale(uint32_t m) {
    return m == 0 ? 127u : (uint32_t)max((int)(m >> 7) - 8 + ((m & 127u) > 96u ? 1 : 0), 1);
}

// One CTA: one block of tokens (blockIdx.x-th from the sequence's unfilled
// block on) and some of its heads.  A group of GW lanes holds R rows of the
// block (8 elements per lane, rounded to bf16 and packed, so that a value is
// the same whether it waited in the ring or came straight from this call);
// rows before lengths[b] come from the ring, the others from k and v.  A full
// block is reduced to its largest magnitude, scaled and written as a page; else
// the new rows go to the ring.  Bound by latency for a round's few rows (11 us a call, the host's
// part of it), by instructions for prompts: 8 x 2048 tokens (8 heads of 128, normed and rotated) take 40 us, 1.9 TB/s, with about 59% of
// the issue slots filled and a barrier in the middle for the block's maximum.  (Angles made of three partial rotations, in f32, took
// 39 us, but turned some keys to the other side of a rounding.)
template <int DT, int R>
__global__ void __launch_bounds__(AP_BT, R <= 4 ? 3 : 2) k_append(const Append P) {
    // cosines, then sines [row of the block][pair]
    extern __shared__ __align__(16) float ct[];
    float* st = ct + P.page * (P.rot / 2);
    __shared__ __align__(16) float wt[128];
    __shared__ uint32_t red[2][AP_BT / 32];
    __shared__ int sh_len;
    const int page = P.page, D = P.D, GW = P.GW;
    const int hgroups = (P.Hkv + P.heads_per_cta - 1) / P.heads_per_cta;
    const int b = blockIdx.y / hgroups, h0 = (blockIdx.y % hgroups) * P.heads_per_cta;
    const int h1 = min(P.Hkv, h0 + P.heads_per_cta);
    const int tid = threadIdx.x, lane = tid & 31, l = lane & (GW - 1), grp = tid / GW;

    // every CTA of the sequence comes to the same verdict; the last to have read
    // the length writes the new one, which may be the same word
    const int cnt = P.num_accepted ? P.num_accepted[b] + 1 : P.W;
    const int slot = P.c.slots ? P.c.slots[b] : b;
    if (tid == 0) sh_len = *reinterpret_cast<const volatile int32_t*>(P.c.lengths + b);
    __syncthreads();
    const int len = sh_len;
    bool bad = cnt < 0 || cnt > P.W || slot < 0 || slot >= P.c.num_slots;
    const int64_t most = (int64_t)P.c.max_pages * page + page - 1;
    bad |= len >= 0 && ((int64_t)len + max(cnt, 0) > most || (int64_t)len + max(cnt, 0) >= SPEC_MAX_CACHE_LEN);
    const int first = len >= 0 ? len / page : 0;
    const int newlen = bad ? 0 : len + cnt;
    if (!bad && len >= 0) {
        const int full = newlen / page;
        for (int j = first + tid; j < full; j += AP_BT) {
            const int id = P.c.page_table[b * P.c.page_table_stride + j];
            bad |= id < 0 || id >= P.c.num_pages;
        }
        if (P.index) {
            for (int i = tid; i < cnt; i += AP_BT) {
                const int r = P.index[(int64_t)b * P.W + i];
                bad |= r < 0 || r >= P.T;
            }
        }
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        __threadfence();
        if (atomicAdd(P.cnt + b, 1u) == gridDim.x * hgroups - 1) {
            P.cnt[b] = 0;
            P.out_lengths[b] = bad && len >= 0 ? -1 : len < 0 ? len : newlen;
            if (bad && len >= 0) atomicOr(P.status, 1u << SPEC_ERR_DEVICE_INPUT);
        }
    }
    if (bad || len < 0 || cnt == 0) return;

    const int last = (newlen - 1) / page;             // last block touched
    int blk = first + (int)blockIdx.x;
    if (blk > last) return;
    // The ring's half of the last block can be the half that still holds the first
    // block's tokens: then the first block's CTA writes the last block too, after
    // it has read them.
    const bool chained = len % page != 0 && newlen % page != 0 && last >= first + 2 && ((last - first) & 1) == 0;
    if (chained && blk == last) return;

    const int groups = AP_BT / GW;                        // D / 8 is 8 or 16: all lanes of a group hold elements
    const float inv_d = 1.f / (float)D;
    const int half = P.rot / 2;
    if (P.kw)
        for (int e = tid; e < D; e += AP_BT) wt[e] = weight_at(P.kw, P.w_f32, e);

    while (true) {
        const int start = blk * page;
        const bool full = start + page <= newlen;
        int page_id = 0;
        if (full) page_id = P.c.page_table[b * P.c.page_table_stride + blk];
        // Each angle on its own, as the norm and rotation call forms it: an appended key is the one that it would have written.
        const int r0 = max(len - start, 0), r1 = min(newlen - start, page);              // the rows that come from k
        for (int j = lane; j < half; j += 32) {
            const float f = P.inv_freq[j];
            for (int r = r0 + (tid >> 5); r < r1; r += AP_BT / 32) {
                const float2 v = cos_sin(start + r, f);
                ct[r * half + j] = v.x;
                st[r * half + j] = v.y;
            }
        }
        // where the rows of the block come from: a row of k and v, the ring (-1), nowhere (-2)
        int from[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = grp + i * groups, t = start + r;
            from[i] = r >= page || t >= newlen ? -2 : t < len ? -1 : P.index ? P.index[(int64_t)b * P.W + (t - len)] : t - len;
        }
        __syncthreads();
        // one (head, keys or values) after the other, the next one's rows on their way
        Quad<DT> raw[R][2];
        const int items = 2 * (h1 - h0);
        auto fetch = [&](int it) {
            const int which = it & 1, h = h0 + (it >> 1);
            const Quads at(l, which ? 0 : P.rot, P.interleaved);
            const int64_t sn = which ? P.v.n : P.k.n;
            const char* src = which ? P.v.p + b * P.v.b + h * P.v.h : P.k.p + b * P.k.b + h * P.k.h;
            const int o0 = at.q0 * 4 * Quad<DT>::ESZ, o1 = at.q1 * 4 * Quad<DT>::ESZ;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                raw[i][0].zero();
                raw[i][1].zero();
                if (from[i] >= 0) {
                    const char* p = src + from[i] * sn;
                    raw[i][0].load(p + o0);
                    raw[i][1].load(p + o1);
                } else if (from[i] == -1) {
                    const char* p = static_cast<const char*>(which ? P.c.v_open : P.c.k_open) +
                                    (((int64_t)slot * P.Hkv + h) * 2 * page + ((start + grp + i * groups) & (2 * page - 1))) * D * 2;
                    raw[i][0].load_bf16(p + 8 * at.q0);
                    raw[i][1].load_bf16(p + 8 * at.q1);
                }
            }
        };
        fetch(0);
        for (int it = 0; it < items; ++it) {
            const int which = it & 1, h = h0 + (it >> 1);
            const Quads at(l, which ? 0 : P.rot, P.interleaved);
            Quad<SPEC_BF16> val[R][2];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int r = grp + i * groups;
                float x[8];
                raw[i][0].get(x);
                raw[i][1].get(x + 4);
                if (which == 0) {                         // rows of the ring are what they are
                    if (P.kw) {
                        const float rs = row_rms(x, GW, inv_d, P.eps);
                        const float4 w0 = *reinterpret_cast<const float4*>(wt + 4 * at.q0), w1 = *reinterpret_cast<const float4*>(wt + 4 * at.q1);
                        if (from[i] >= 0) {
                            x[0] = x[0] * rs * w0.x; x[1] = x[1] * rs * w0.y; x[2] = x[2] * rs * w0.z; x[3] = x[3] * rs * w0.w;
                            x[4] = x[4] * rs * w1.x; x[5] = x[5] * rs * w1.y; x[6] = x[6] * rs * w1.z; x[7] = x[7] * rs * w1.w;
                        }
                    }
                    if (at.turns && from[i] >= 0)
                        row_rotate(x, *reinterpret_cast<const float4*>(ct + r * half + 4 * l),
                                   *reinterpret_cast<const float4*>(st + r * half + 4 * l), P.interleaved);
                }
                val[i][0].set(x);
                val[i][1].set(x + 4);
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(val[i][0].a.x & 0x7fff7fffu, val[i][0].a.y & 0x7fff7fffu),
                                         __vmaxu2(val[i][1].a.x & 0x7fff7fffu, val[i][1].a.y & 0x7fff7fffu)));
            }
            if (it + 1 < items) fetch(it + 1);
            if (!full) {
                char* ring = static_cast<char*>(which ? P.c.v_open : P.c.k_open) + ((int64_t)slot * P.Hkv + h) * 2 * page * D * 2;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (from[i] >= 0) {
                        char* p = ring + (int64_t)((start + grp + i * groups) & (2 * page - 1)) * D * 2;
                        val[i][0].store(p + 8 * at.q0);
                        val[i][1].store(p + 8 * at.q1);
                    }
                }
                continue;
            }
            m = max(m & 0xffffu, m >> 16);                // bits of the largest magnitude
            const bool odd = m >= 0x7f80u;                // something here is not finite
            if (odd) {
                m = 0;
                for (int i = 0; i < R; ++i)
                    for (int u = 0; u < 8; ++u) {
                        const uint2 w = val[i][u >> 2].a;
                        const uint32_t a = ((u & 2 ? w.y : w.x) >> (u & 1 ? 16 : 0)) & 0x7fffu;
                        if (a < 0x7f80u) m = max(m, a);
                    }
            }
            m = __reduce_max_sync(FULL, m);
            if (lane == 0) red[it & 1][tid >> 5] = m;
            __syncthreads();                              // of the two rows of `red`, the other is still being read
            m = red[it & 1][0];
#pragma unroll
            for (int w = 1; w < AP_BT / 32; ++w) m = max(m, red[it & 1][w]);
            const uint32_t sc = block_scale(m);
            const float inv = __uint_as_float((254u - sc) << 23);
            const int64_t ph = (int64_t)page_id * P.Hkv + h;
            if (tid == 0) (which ? P.c.v_scale : P.c.k_scale)[ph] = __uint_as_float(sc << 23);
            char* dst = static_cast<char*>(which ? P.c.v_pages : P.c.k_pages) + ph * page * D;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int r = grp + i * groups;
                if (r >= page) continue;
                float x[8];
                val[i][0].get(x);
                val[i][1].get(x + 4);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    x[u] *= inv;
                    if (odd && !(fabsf(x[u]) <= 448.f)) x[u] = __int_as_float(0x7fffffff);
                }
                *reinterpret_cast<uint32_t*>(dst + (int64_t)r * D + 4 * at.q0) = pack_e4m3(x[0], x[1]) | pack_e4m3(x[2], x[3]) << 16;
                *reinterpret_cast<uint32_t*>(dst + (int64_t)r * D + 4 * at.q1) = pack_e4m3(x[4], x[5]) | pack_e4m3(x[6], x[7]) << 16;
            }
        }
        if (!chained || blk != first) break;
        __syncthreads();                                  // the first block's ring rows and angles have been read
        blk = last;
    }
}

template <int DT, int R>
spec_status launch_append_rows(const Append& P, dim3 grid, cudaStream_t st) {
    const size_t smem = (size_t)P.page * (P.rot / 2) * sizeof(float2);       // up to 64 KB
    // asked for whatever this call needs: the kernel's static shared memory counts towards the 48 KB too
    static std::atomic<uint64_t> done{0};
    if (const spec_status s = sv_host::allow_smem(reinterpret_cast<const void*>(k_append<DT, R>), "k_append", 64 * 1024, done)) return s;
    k_append<DT, R><<<grid, AP_BT, smem, st>>>(P);
    return sv_host::launched("k_append");
}

template <int DT>
spec_status launch_append(const Append& P, dim3 grid, int rows, cudaStream_t st) {
    return rows <= 1 ? launch_append_rows<DT, 1>(P, grid, st)
           : rows == 2 ? launch_append_rows<DT, 2>(P, grid, st)
           : rows == 4 ? launch_append_rows<DT, 4>(P, grid, st) : launch_append_rows<DT, 8>(P, grid, st);
}

int group_width(int D) {
    int w = 1;
    while (w < D / 8) w *= 2;
    return w;
}

spec_status check_dims(int B, int N) {
    if (B < 0) return sv_host::fail(SPEC_ERR_INVALID_ARG, "B %d < 0", B);
    if (N < 1 || N > SPEC_MAX_NODES)
        return sv_host::fail(SPEC_ERR_INVALID_ARG, "N %d outside [1, %d]", N, SPEC_MAX_NODES);
    return SPEC_OK;
}

spec_status check_rotation(int D, int rot, int interleaved, const float* inv_freq, spec_dtype wdt, float eps) {
    if (rot < 0 || rot > D || rot % 16 != 0)
        return sv_host::fail(SPEC_ERR_INVALID_ARG, "rot_dim %d is not a multiple of 16 in [0, D %d]", rot, D);
    if (rot && !inv_freq) return sv_host::fail(SPEC_ERR_INVALID_ARG, "inv_freq is NULL");
    if (interleaved != 0 && interleaved != 1) return sv_host::fail(SPEC_ERR_INVALID_ARG, "interleaved is not 0 or 1");
    if (wdt != SPEC_F32 && wdt != SPEC_BF16) return sv_host::fail(SPEC_ERR_INVALID_ARG, "unknown weight dtype %d", (int)wdt);
    if (!(eps >= 0.f) || eps > 3.402823466e38f) return sv_host::fail(SPEC_ERR_INVALID_ARG, "eps is not a finite value >= 0");
    return SPEC_OK;
}

// An output's rows are apart: a broadcast one would be written by several CTAs at once.
spec_status check_apart(const char* what, const int64_t* strides, int B, int N, int H, int D) {
    const int dims[3] = {B, N, H};
    for (int i = 0; i < 3; ++i)
        if (dims[i] > 1 && strides[i] < D && strides[i] > -D)
            return sv_host::fail(SPEC_ERR_INVALID_ARG, "%s: stride %d (%lld elements) is less than a row of %d", what, i,
                                 (long long)strides[i], D);
    return SPEC_OK;
}

spec_status check_weight(const char* what, const void* w) {
    if (w && ((uintptr_t)w & 15u) != 0) return sv_host::fail(SPEC_ERR_INVALID_ARG, "%s not 16-byte aligned", what);
    return SPEC_OK;
}

}  // namespace

namespace sv_host {

spec_status check_cache_ws(void* ws, size_t bytes, size_t need) {
    if (!ws) return fail(SPEC_ERR_WORKSPACE, "workspace is NULL");
    if (((uintptr_t)ws & 255u) != 0) return fail(SPEC_ERR_WORKSPACE, "workspace not 256-byte aligned");
    if (bytes < need) return fail(SPEC_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
    return SPEC_OK;
}

spec_status check_cache(const spec_kv_cache* c, int B) {
    if (!c) return fail(SPEC_ERR_INVALID_ARG, "cache is NULL");
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(SPEC_ERR_INVALID_ARG, "cache: head_dim %d is not 64 or 128", c->head_dim);
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return fail(SPEC_ERR_INVALID_ARG, "cache: page_size %d is not 16, 32, 64 or 128", c->page_size);
    if (c->kv_heads < 1 || c->kv_heads > SPEC_MAX_HEADS)
        return fail(SPEC_ERR_INVALID_ARG, "cache: kv_heads %d outside [1, %d]", c->kv_heads, SPEC_MAX_HEADS);
    if (c->max_pages < 0 || c->page_table_stride < c->max_pages)
        return fail(SPEC_ERR_INVALID_ARG, "cache: max_pages %d, page_table_stride %lld", c->max_pages,
                    (long long)c->page_table_stride);
    if (c->num_pages < 0 || c->num_pages > INT32_MAX)
        return fail(SPEC_ERR_INVALID_ARG, "cache: num_pages %lld", (long long)c->num_pages);
    if (c->num_pages * c->kv_heads * c->page_size > INT32_MAX)       // a row is a 32-bit coordinate of the tensor copies
        return fail(SPEC_ERR_INVALID_ARG, "cache: %lld pages of %d heads x %d tokens are more than 2^31 - 1 rows",
                    (long long)c->num_pages, c->kv_heads, c->page_size);
    if (c->num_slots < 0 || (!c->slots && c->num_slots < B))
        return fail(SPEC_ERR_INVALID_ARG, "cache: %d slots for %d sequences", c->num_slots, B);
    if (B > 0 && !c->lengths) return fail(SPEC_ERR_INVALID_ARG, "cache: lengths are NULL");
    if (B > 0 && c->max_pages > 0 && !c->page_table) return fail(SPEC_ERR_INVALID_ARG, "cache: page_table is NULL");
    const void* data[4] = {c->k_pages, c->v_pages, c->k_open, c->v_open};
    for (int i = 0; i < 4; ++i) {
        const bool needed = i < 2 ? c->num_pages > 0 : c->num_slots > 0;
        if (needed && !data[i]) return fail(SPEC_ERR_INVALID_ARG, "cache: %s NULL", i < 2 ? "pages are" : "ring is");
        if (((uintptr_t)data[i] & 15u) != 0)
            return fail(SPEC_ERR_INVALID_ARG, "cache: %s not 16-byte aligned", i < 2 ? "pages" : "ring");
    }
    if (c->num_pages > 0 && (!c->k_scale || !c->v_scale)) return fail(SPEC_ERR_INVALID_ARG, "cache: scales are NULL");
    return SPEC_OK;
}

}  // namespace sv_host

using sv_host::fail;

extern "C" {

spec_status spec_tree_plan(int B, int N, int max_depth, const int32_t* parents, const int32_t* lengths,
                           int32_t* out_positions, int32_t* out_ancestors,
                           void* workspace, size_t workspace_bytes, void* stream) {
    sv_host::Range range("spec_tree_plan");
    if (spec_status s = check_dims(B, N)) return s;
    if (max_depth < 0 || max_depth > SPEC_MAX_DEPTH)
        return fail(SPEC_ERR_INVALID_ARG, "max_depth %d outside [0, %d]", max_depth, SPEC_MAX_DEPTH);
    if (B == 0) return SPEC_OK;
    if (!lengths || !out_positions || !out_ancestors) return fail(SPEC_ERR_INVALID_ARG, "a pointer is NULL");
    if (spec_status s = sv_host::check_cache_ws(workspace, workspace_bytes, sv_host::CACHE_WS_PARTIAL)) return s;
    const int bt = (N + 31) / 32 * 32;
    k_tree_plan<<<B, bt, 0, static_cast<cudaStream_t>(stream)>>>(N, max_depth, parents, lengths, out_positions,
                                                                 reinterpret_cast<uint32_t*>(out_ancestors),
                                                                 static_cast<unsigned*>(workspace));
    return sv_host::launched("k_tree_plan");
}

spec_status spec_qk_norm_rope(int B, int N, int q_heads, int kv_heads, int D,
                              const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                              spec_dtype dt, const int32_t* positions,
                              const float* inv_freq, int rot_dim, int interleaved,
                              const void* q_weight, const void* k_weight, spec_dtype wdt, float eps,
                              void* q_out, const int64_t* q_out_strides,
                              void* k_out, const int64_t* k_out_strides, void* stream) {
    sv_host::Range range("spec_qk_norm_rope");
    if (B < 0 || N < 1 || (int64_t)B * N > INT32_MAX)
        return fail(SPEC_ERR_INVALID_ARG, "B %d, N %d", B, N);
    if (q_heads < 1 || q_heads > SPEC_MAX_HEADS || kv_heads < 0 || kv_heads > SPEC_MAX_HEADS)
        return fail(SPEC_ERR_INVALID_ARG, "q_heads %d, kv_heads %d", q_heads, kv_heads);
    if (D < 8 || D > 256 || D % 8 != 0) return fail(SPEC_ERR_INVALID_ARG, "D %d is not a multiple of 8 in [8, 256]", D);
    if (dt != SPEC_F32 && dt != SPEC_BF16) return fail(SPEC_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (spec_status s = check_rotation(D, rot_dim, interleaved, inv_freq, wdt, eps)) return s;
    if (spec_status s = check_weight("q_weight", q_weight)) return s;
    if (spec_status s = check_weight("k_weight", k_weight)) return s;
    if (B == 0) return SPEC_OK;
    if (!positions) return fail(SPEC_ERR_INVALID_ARG, "positions are NULL");
    NormRope P{};
    const int esz = dt == SPEC_F32 ? 4 : 2;
    if (spec_status s = sv_host::make_rows("q", q, q_strides, B, N, q_heads, esz, &P.q)) return s;
    if (spec_status s = sv_host::make_rows("q_out", q_out, q_out_strides, B, N, q_heads, esz, &P.qo)) return s;
    if (spec_status s = check_apart("q_out", q_out_strides, B, N, q_heads, D)) return s;
    if (kv_heads) {
        if (spec_status s = sv_host::make_rows("k", k, k_strides, B, N, kv_heads, esz, &P.k)) return s;
        if (spec_status s = sv_host::make_rows("k_out", k_out, k_out_strides, B, N, kv_heads, esz, &P.ko)) return s;
        if (spec_status s = check_apart("k_out", k_out_strides, B, N, kv_heads, D)) return s;
    }
    P.B = B; P.N = N; P.Hq = q_heads; P.Hk = kv_heads; P.D = D; P.rot = rot_dim; P.interleaved = interleaved;
    P.GW = group_width(D);
    P.pos = positions; P.inv_freq = inv_freq;
    P.qw = static_cast<const char*>(q_weight);
    P.kw = static_cast<const char*>(k_weight);
    P.w_f32 = wdt == SPEC_F32;
    P.eps = eps;
    // few tokens: their heads over several CTAs
    const int heads = q_heads + kv_heads, groups = NR_BT / P.GW, tokens = B * N;
    int split = 4 * sv_host::num_sms() / tokens;
    const int most = (heads + groups - 1) / groups;
    split = split < 1 ? 1 : split > most ? most : split;
    const dim3 grid(tokens, split);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dt == SPEC_F32) k_norm_rope<SPEC_F32><<<grid, NR_BT, 0, st>>>(P);
    else k_norm_rope<SPEC_BF16><<<grid, NR_BT, 0, st>>>(P);
    return sv_host::launched("k_norm_rope");
}

spec_status spec_kv_append(int B, int T, int width, const spec_kv_cache* cache,
                           const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides,
                           spec_dtype dt, const int32_t* num_accepted, const int32_t* accept_index,
                           const float* inv_freq, int rot_dim, int interleaved,
                           const void* k_weight, spec_dtype wdt, float eps,
                           int32_t* out_lengths,
                           void* workspace, size_t workspace_bytes, void* stream) {
    sv_host::Range range("spec_kv_append");
    if (B < 0 || T < 1 || T > (1 << 20) || width < 1 || width > (1 << 20))
        return fail(SPEC_ERR_INVALID_ARG, "B %d, T %d, width %d", B, T, width);
    if (!accept_index && width > T) return fail(SPEC_ERR_INVALID_ARG, "width %d > T %d without accept_index", width, T);
    if (dt != SPEC_F32 && dt != SPEC_BF16) return fail(SPEC_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
    if (spec_status s = sv_host::check_cache(cache, B)) return s;
    const int D = cache->head_dim, page = cache->page_size, Hkv = cache->kv_heads;
    if (spec_status s = check_rotation(D, rot_dim, interleaved, inv_freq, wdt, eps)) return s;
    if (spec_status s = check_weight("k_weight", k_weight)) return s;
    if (B == 0) return SPEC_OK;
    if (!out_lengths) return fail(SPEC_ERR_INVALID_ARG, "out_lengths is NULL");
    Append P{};
    const int esz = dt == SPEC_F32 ? 4 : 2;
    if (spec_status s = sv_host::make_rows("k", k, k_strides, B, T, Hkv, esz, &P.k)) return s;
    if (spec_status s = sv_host::make_rows("v", v, v_strides, B, T, Hkv, esz, &P.v)) return s;
    if (B > sv_host::CACHE_MAX_B) return fail(SPEC_ERR_INVALID_ARG, "B %d > %d", B, sv_host::CACHE_MAX_B);
    if (spec_status s = sv_host::check_cache_ws(workspace, workspace_bytes, sv_host::CACHE_WS_PARTIAL)) return s;
    char* ws = static_cast<char*>(workspace);
    P.B = B; P.T = T; P.W = width; P.Hkv = Hkv; P.D = D; P.page = page; P.rot = rot_dim; P.interleaved = interleaved;
    P.w_f32 = wdt == SPEC_F32;
    P.GW = group_width(D);
    P.c = *cache;
    P.num_accepted = num_accepted; P.index = accept_index; P.inv_freq = inv_freq;
    P.kw = static_cast<const char*>(k_weight);
    P.eps = eps;
    P.out_lengths = out_lengths;
    P.status = reinterpret_cast<unsigned*>(ws + sv_host::CACHE_WS_STATUS);
    P.cnt = reinterpret_cast<unsigned*>(ws + sv_host::CACHE_WS_SEQ);
    const int blocks = (page - 1 + width - 1) / page + 1;          // touched at most
    // a CTA takes several heads (they share the angles) once there are CTAs enough for four per SM: with the angles made of partial
    // rotations 8 x 2048 tokens took 43 us with eight, 39 with four, 45 with three; 1 x 2048 13.3 us with each of them, 15 with two
    // heads to a CTA
    const long long units = (long long)blocks * B * Hkv;
    long long per = (units + 4LL * sv_host::num_sms() - 1) / (4LL * sv_host::num_sms());
    P.heads_per_cta = (int)(per < 1 ? 1 : per > Hkv ? Hkv : per);
    const long long ys = (long long)B * ((Hkv + P.heads_per_cta - 1) / P.heads_per_cta);
    if (ys > 65535) return fail(SPEC_ERR_INVALID_ARG, "B * kv_heads = %lld is above 65535 rows of CTAs", ys);
    const dim3 grid(blocks, (unsigned)ys);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rows = page / (AP_BT / P.GW);                        // block rows per group of lanes: 0 (some idle) to 8
    if (dt == SPEC_F32) return launch_append<SPEC_F32>(P, grid, rows, st);
    return launch_append<SPEC_BF16>(P, grid, rows, st);
}

}  // extern "C"
