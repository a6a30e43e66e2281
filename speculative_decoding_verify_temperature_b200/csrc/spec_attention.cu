// spec_attention.cu -- attention of the nodes of draft trees over the paged
// 8-bit cache and each other.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "cache_device.cuh"
#include "internal.h"

using namespace svc;

namespace {

constexpr int TILE = 128;                 // keys of one step
constexpr float NEG_INF = -INFINITY;
constexpr float LN2 = 0.69314718055994530942f;

struct Att {
    int B, N, Hq, Hkv, G, page, pshift, R;   // page = 1 << pshift; R = N * G rows of a kv head
    int mtiles;                           // items per (sequence, kv head)
    int over;                             // what an item costs beside its tiles, in tiles
    sv_host::Rows q, k, v;
    spec_kv_cache c;
    const uint32_t* anc;                  // nullable: chains
    float scale;                          // scale * log2(e)
    char* out;
    float* lse;
    unsigned* status;
    unsigned wait_tries;                  // polls of the first wait for copied bytes
    struct Cut* cut;                      // [gridDim.x] the item that a CTA begins and does not end
    float* partial;                       // [gridDim.x][2][rows of an item][D + 3]
};

// An item whose tiles several CTAs share: they leave partial results, the CTA that
// begins it in slot 1 of its workspace and those after it in slot 0 of theirs.
struct Cut {
    int b, h, mt, parts;                  // parts = 0: none
};

// ----------------------------------------------------------------------------- the work and its split

// The keys of a sequence: `full` cached tokens in 8-bit blocks, then a tail of
// `open` tokens of the unfilled block and the N nodes.  Each part is cut into
// tiles of TILE keys.
struct Seq {
    int len, slot, full, open, nct, ntiles;
    bool bad;
};

__device__ __forceinline__ Seq seq_of(const Att& P, int b) {
    Seq s;
    s.len = P.c.lengths[b];
    s.slot = P.c.slots ? P.c.slots[b] : b;
    const int64_t most = (int64_t)P.c.max_pages * P.page + P.page - 1;
    s.bad = s.len >= 0 && (s.len > most || s.len >= SPEC_MAX_CACHE_LEN || s.slot < 0 || s.slot >= P.c.num_slots);
    const bool live = s.len >= 0 && !s.bad;
    s.full = live ? s.len >> P.pshift << P.pshift : 0;
    s.open = live ? s.len - s.full : 0;
    s.nct = (s.full + TILE - 1) / TILE;
    s.ntiles = s.nct + (s.open + P.N + TILE - 1) / TILE;
    if (!live) s.nct = 0, s.ntiles = 1;   // one step that writes the rows' zeros or NaN
    return s;
}

// The items (sequence, kv head, rows), in that order, are one line: each takes
// `over` units (its queries, its tail and its results) and one for each of its
// tiles.  Every CTA takes an equal stretch of the line, whatever the lengths are.
// An item whose tiles a stretch border cuts leaves partial results, which a second
// kernel puts together.
struct Stretch {
    long long lo, hi, total;              // units
    int ctas;                             // CTAs that share the line: each has at least one unit
    int b;                                // sequence of unit lo
    long long b_lo;                       // first unit of that sequence
};

__device__ __forceinline__ long long stretch_at(long long total, int cta, int ctas) { return total * cta / ctas; }
// CTA that holds unit x.
__device__ __forceinline__ int cta_of(long long x, long long total, int ctas) {
    int c = (int)(x * ctas / total);
    while (stretch_at(total, c + 1, ctas) <= x) ++c;
    while (stretch_at(total, c, ctas) > x) --c;
    return c;
}

// All threads of the CTA (BT of them).  Two passes over the lengths: the total, then the sequence
// where the stretch begins.
template <int BT>
__device__ Stretch find_stretch(const Att& P) {
    __shared__ long long wsum[BT / 32 + 1];
    __shared__ int hit_b;
    __shared__ long long hit_lo;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int items = P.Hkv * P.mtiles;
    Stretch s{};
    long long mine = 0, first = 0;
    for (int b = tid; b < P.B; b += BT) {
        const long long n = (long long)(seq_of(P, b).ntiles + P.over) * items;
        if (b == tid) first = n;
        mine += n;
    }
    long long sum = mine;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    if (lane == 0) wsum[warp] = sum;
    __syncthreads();
    for (int w = 0; w < BT / 32; ++w) s.total += wsum[w];
    s.ctas = (int)min((long long)gridDim.x, s.total);
    if ((int)blockIdx.x >= s.ctas) return s;               // the same in every thread; lo = hi
    s.lo = stretch_at(s.total, blockIdx.x, s.ctas);
    s.hi = stretch_at(s.total, blockIdx.x + 1, s.ctas);
    long long before = 0;
    for (int base = 0; base < P.B; base += BT) {
        const int b = base + tid;
        const long long n = base == 0 ? first : b < P.B ? (long long)(seq_of(P, b).ntiles + P.over) * items : 0;
        long long inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += up;
        }
        __syncthreads();
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        long long off = before, all = 0;
        for (int w = 0; w < BT / 32; ++w) {
            if (w < warp) off += wsum[w];
            all += wsum[w];
        }
        inc += off;
        if (s.lo < inc && s.lo >= inc - n) {
            hit_b = b;
            hit_lo = inc - n;
        }
        before += all;
        if (before > s.lo) break;
    }
    __syncthreads();
    s.b = hit_b;
    s.b_lo = hit_lo;
    return s;
}

// A CTA's part of one item: at least one of its tiles.
struct Seg {
    Seq q;
    int b, h, mt;
    int t0, t1;                           // tiles of the item
    long long item_lo;                    // the item's first unit on the line
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == q.ntiles; }
};

struct SegIter {
    Stretch s;
    long long at, item_lo;
    int b, item;
    Seq q;
    __device__ __forceinline__ void begin(const Att& P, const Stretch& st) {
        s = st;
        at = st.lo;
        b = st.b;
        if (at < s.hi) {
            q = seq_of(P, b);
            item = (int)((at - st.b_lo) / (q.ntiles + P.over));
            item_lo = st.b_lo + (long long)item * (q.ntiles + P.over);
        }
    }
    __device__ __forceinline__ bool next(const Att& P, Seg& g) {
        while (at < s.hi) {
            if (item == P.Hkv * P.mtiles) {
                item = 0;
                q = seq_of(P, ++b);
            }
            const int units = q.ntiles + P.over;
            g.q = q;
            g.b = b;
            g.h = item / P.mtiles;
            g.mt = item - g.h * P.mtiles;
            g.item_lo = item_lo;
            g.t0 = max((int)(at - item_lo) - P.over, 0);
            g.t1 = (int)min((long long)units, s.hi - item_lo) - P.over;
            ++item;
            at = item_lo += units;
            if (g.t1 > g.t0) return true;                 // else the stretch ends before the item's first tile
        }
        return false;
    }
};

// CTAs that hold tiles of the item which this CTA begins and does not end.
__device__ __forceinline__ int parts_of(const Att& P, const Seg& g, const Stretch& st, int cta) {
    return cta_of(g.item_lo + P.over + g.q.ntiles - 1, st.total, st.ctas) - cta + 1;
}

// 32 bits of the mask of node n over the tail's keys [e0, e0 + 32): the open
// tokens are seen by every node, node m by the rows whose mask holds it.
__device__ __forceinline__ uint32_t tail_bits(const Att& P, int b, int n, int open, int e0) {
    uint32_t bits = 0;
    if (e0 < open) bits = open - e0 >= 32 ? 0xffffffffu : (1u << (open - e0)) - 1u;
    const int m0 = e0 - open;             // node of bit 0 (negative: an open token)
    if (m0 > -32 && m0 < P.N) {
        uint32_t nodes;
        if (P.anc) {
            const int W = (P.N + 31) / 32;
            const uint32_t* a = P.anc + ((int64_t)b * P.N + n) * W;
            const int w = m0 >> 5, sh = m0 & 31;           // arithmetic shift: w = -1 for m0 < 0
            const uint32_t lo = w >= 0 ? __ldg(a + w) : 0u, hi = w + 1 < W ? __ldg(a + w + 1) : 0u;
            nodes = __funnelshift_r(lo, hi, sh);
        } else {
            const int last = n - m0;      // nodes 0..n
            nodes = last < 0 ? 0u : last >= 31 ? 0xffffffffu : (2u << last) - 1u;
            if (m0 < 0) nodes &= 0xffffffffu << -m0;
        }
        const int left = P.N - m0;
        if (left < 32) nodes &= (1u << left) - 1u;
        bits |= nodes;
    }
    return bits;
}

// ----------------------------------------------------------------------------- tensor-core kernel (tcgen05)

// Roles of the CTA's warps: 0-3 and 4-7 the softmax of one stream each, 8-15 make
// operands (f16 values from e4m3 bytes, queries, the tail), 16 issues the matrix
// instructions, 17 copies pages to shared memory, 18 gathers the
// pages' scales, 19 nothing.
//
// An item holds up to 256 rows.  With more than 128 the two streams are its two
// halves and both take every tile; with 128 or fewer both streams hold the same
// rows and take the tiles in turn, and their sums are joined at the end.  While
// one stream's softmax works on its scores, the tensor cores work for the other.
//
//   S_i = Q_i K^T    e4m3 operands, f32 in tensor memory
//   P_i              f16, over S_i's columns
//   O_i += P_i V     f16, P from tensor memory, V from shared memory
//
// Keys go to the tensor cores as the cache holds them: a swizzled tensor copy
// brings a page's bytes to where the matrix instruction reads them.  The other
// side is split: a bf16 row of q, divided by a power of two that brings its
// largest magnitude to [128, 256), is the sum of two e4m3 rows (four bits of
// its eight each; an element below 2^-9 of the largest is rounded at 2^-18 of it), so a score is
// two products.  The tail's keys are split the same way, four products.
// Values are turned into f16, which holds every e4m3 value; the tail's rows are divided by a power of two that brings their
// largest magnitude to [1, 2), so elements below 2^-17 of it are rounded at 2^-25 of it.  Brought higher, rows would keep more of
// themselves but weigh the rounding of their P more, which are that much smaller: the bound below, 2^-36 of the leading
// weight times |v| / s_v for each key, would be passed (it was, with [2^14, 2^15)).
//
// The scales come back in f32: with a_j the key's scale times the row's and
// s_v,j the value's, x_j = S_j a_j is the score in base 2 and
//   w_j = x_j + log2 s_v,j,  M = max w_j,  P_j = 2^(w_j - M),
//   O = sum P_j v_j,  l = sum P_j / s_v,j,  out = O / l.
// M follows the weight with which a value enters O, so that f16 holds the
// leading P whatever the blocks' scales are.  M is kept a whole number (rounded up),
// so that bringing earlier P to a larger one only moves their exponents, and it
// is changed only when it grows by more than 3; P_BIAS lifts P to at most 2^15, and
// the leading one to 2^11 or more: f16's smallest step is 2^-35 of it.
//
// l stands relative to the same M, although it has nothing to do with the values: P_j / s_v,j is 2^(x_j - M + P_BIAS),
// which leaves the range of f32 where M is more than 100 or so away from the largest x_j.  With every s_v,j within
// [FAR_LO, FAR_HI] it is at most 43 away, and what f32 drops of l lies 2^-55 below its leading part.  From the first tile with
// another scale on, a row's l is summed from exponentials of its own, 2^(x_j - r), with r a whole number that
// follows the largest x_j ("far"; r = M - P_BIAS otherwise), and out = O / l 2^(M - P_BIAS - r).  That costs a second
// exponential per key, in code that trained values do not reach; the others pay for it in an item's own steps (64 chains of 6
// over ragged lengths up to 4096 198 -> 204 us; 32 trees of 64 and one tree of 32, see below, as before).
//
// Measured (B200, D = 128, 64 query on 8 kv heads): 32 trees of 64 nodes over ragged lengths up to 8192 550 us, 630 TFLOP/s;
// 64 chains of 6 over ragged lengths up to 4096 206 us; one tree of 32 over 131072 tokens (32 query heads of 64) 106 us.  Bound by the
// chain of one stream's steps, about 5400 cycles a tile: softmax 3100 (its own warp's latencies: MUFU a third busy), the
// product with values 700, the scores of the next tile 850, barriers the rest; the two streams run side by side and tensor
// memory (S0 S1 O0 O1 fill it at D = 128) has no room for a third.  An item costs another 25000 cycles or so.  Tried and slower:
// a second warp for the matrix instructions (204 -> 220 us: what waits is the chain, not the warp), the scores in two
// halves of 64 keys, the first beside the product before (550 -> 690 us: an instruction takes about 90 cycles whatever its N).
constexpr int TC_SOFTMAX = 256, TC_CONV = 256, TC_BT = 640;
constexpr int TC_W_CONV = 8, TC_W_MMA = 16, TC_W_COPY = 17, TC_W_SCALE = 18;
constexpr int TC_META = 4;                // tiles whose scales are kept
constexpr float P_BIAS = 12.f, M_SLACK = 3.f;
constexpr float FAR_LO = 0x1p-40f, FAR_HI = 0x1p40f, R_SLACK = 20.f;
__device__ __forceinline__ bool is_far(float s) { return !(s >= FAR_LO && s <= FAR_HI); }
__device__ __forceinline__ bool is_far_exp(int e) { return e < -40 || e > 40; }

template <int D> struct Tc {
    static constexpr int HALVES = D / 64;                 // 128-byte rows of 64 f16
    static constexpr uint32_t HALF = 128 * 128;           // 128 such rows
    static constexpr uint32_t V_B = HALVES * HALF;        // f16 values of a tile
    static constexpr uint32_t RAW_B = TILE * D;           // e4m3 rows of a tile
    static constexpr uint32_t Q_B = TILE * 2 * D;         // both e4m3 rows of 128 queries
    static constexpr int KR = D == 128 ? 3 : 6, VR = D == 128 ? 2 : 4;   // units of keys, of value bytes
    static constexpr uint32_t Q = 0, K = Q + 2 * Q_B, RAW = K + KR * RAW_B, V = RAW + VR * RAW_B, END = V + 2 * V_B;
    static constexpr int O_COL = 256;                     // tensor memory columns: S0 S1 (128 each), O0 O1 (D each)
};
struct TcShared {
    // per key (tail) or group of 16 (cached): a, log2 s_v, 1 / s_v; of a far tile: a, +inf, -1, log2 s_v
    float meta[TC_META][4][TILE];
    float rq[4][256];                                     // per row: its power of two * scale * log2(e)
    float xm[2][TILE], xl[2][TILE];                       // M and l of the streams that are joined
    float far[3][2][TILE];                                // M, l and r of far rows
    int far_tail;                                         // 1 + the last tail tile with a far key
    uint32_t bad_v[4][12];                                // tail keys whose value is not finite
    int bad_seg[8];                                       // 1 + segment that met a bad page
    uint64_t kf[6], ke[6], rf[4], re[4], vf[2], ve[2], mf[TC_META], me[TC_META], sf[2], pf[2], pv[2], qf, qe, drain;
    uint32_t tmem;
    int abort;
};
// 1 KB of alignment slack; at least what keeps a second CTA, and its tensor memory, off the SM
template <int D> constexpr size_t tc_smem() {
    const size_t need = Tc<D>::END + sizeof(TcShared) + 1024;
    return need > 120 * 1024 ? need : 120 * 1024;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// What a sum relative to 2^from counts relative to 2^to >= 2^from (-inf: an empty sum, whose NaN stays).
__device__ __forceinline__ float moved(float from, float to) { return from == NEG_INF ? (to == NEG_INF ? 1.f : 0.f) : ex2(from - to); }
// What takes O to an output is 1 / l and 2^g, g = M - P_BIAS - r, 0 unless the row is far.  2^(g / 2), twice, stays in f32's range.
__device__ __forceinline__ float lift_of(float m, float r) { return m == NEG_INF ? 0.f : m - P_BIAS - r; }
__device__ __forceinline__ float half_exp2(float g) { return ex2(0.5f * g); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four e4m3 bytes to f16 (exact), bytes (0, 1) and (2, 3).
__device__ __forceinline__ uint2 e4m3_f16(uint32_t w) {
    uint2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}" : "=r"(r.x), "=r"(r.y) : "r"(w));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint2 v) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" :: "r"(a), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two f32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Barriers.  Every wait is bounded: when one gives up, the CTA's `abort` is set
// and all waits return at once; every role then runs through its (finite) loops
// with whatever is there, the rows' results become NaN and the status word says why.  What a role arrives with after such a
// wait comes after `abort`, so whoever takes it for the real thing finds `abort` set at the rows' end.  Barriers that count
// arrivals alone stay in order whatever arrives; those that count bytes too (kf, rf) would not, so nobody arrives there and no copy is
// sent after a failed wait.
constexpr unsigned WAIT_TRIES = 1u << 24;
constexpr unsigned long long WAIT_NS = 1000000000ull;
__device__ __forceinline__ void bar_init(uint64_t* b, unsigned n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(smem_u32(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* b) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void copy4(const float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrives once this thread's copy4()s have landed.
__device__ __forceinline__ void copy4_arrive(uint64_t* b) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(b)) : "memory");
}
// Rows [row, row + box) of the tensor map's 8-bit matrix, all columns, swizzled.
__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap* map, int row, uint64_t* b) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(0), "r"(row), "r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool aborted(const TcShared& sh) { return *reinterpret_cast<const volatile int*>(&sh.abort) != 0; }
__device__ __forceinline__ unsigned long long global_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __noinline__ bool bar_wait_slow(uint64_t* b, uint32_t parity, volatile int* abort, unsigned tries = WAIT_TRIES) {
    if (abort && *abort) return false;
    const unsigned long long t0 = global_ns();
    for (unsigned i = 0; i < tries; ++i) {
        if (bar_try(b, parity)) return true;
        if ((i & 63) == 63) {
            if (abort && *abort) return false;
            if (global_ns() - t0 > WAIT_NS) break;
        }
    }
    return false;
}
// Whole warps call it: lanes may leave the polls one after the other, and what follows (tensor memory accesses, elected
// issue) wants them together.
__device__ __forceinline__ void bar_wait(uint64_t* b, uint32_t parity, TcShared& sh) {
    if (!bar_try(b, parity) && !bar_wait_slow(b, parity, &sh.abort)) *reinterpret_cast<volatile int*>(&sh.abort) = 1;
    __syncwarp();
}
// The first wait for bytes that were copied: `tries` polls (a testing hook: 0 gives up at once).
__device__ __forceinline__ void bar_wait_copy(uint64_t* b, uint32_t parity, TcShared& sh, unsigned tries) {
    if (tries == 0 || (!bar_try(b, parity) && !bar_wait_slow(b, parity, &sh.abort, tries))) *reinterpret_cast<volatile int*>(&sh.abort) = 1;
    __syncwarp();
}

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// The warp that issues matrix instructions stays together and one elected lane issues: what all lanes compute alike
// stays in uniform registers, where these instructions take their operands from.  (From one lane's branch each operand
// was moved there first: 170 cycles an instruction.)
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void tc_commit(uint64_t* b, uint32_t lead) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 :: "r"(smem_u32(b)), "r"(lead) : "memory");
}
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t lead) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(lead) : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t lead) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(lead) : "memory");
}
// The registers are operands, so that nothing that uses them comes before the wait.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_ld32(uint32_t a, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(a));
}
__device__ __forceinline__ void tc_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15};"
                 :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                    "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
                 : "memory");
}

// Sixteen columns, waited for.
__device__ __forceinline__ void tc_ld16(uint32_t a, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(a) : "memory");
}
// Eight columns, waited for.
__device__ __forceinline__ void tc_ld8(uint32_t a, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a) : "memory");
}
__device__ __forceinline__ void tc_ld4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(a) : "memory");
}
__device__ __forceinline__ void tc_st4(uint32_t a, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};"
                 :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(a) : "memory");
}

// Shared-memory operand descriptor: rows of ROW bytes swizzled over ROW bytes (128
// or 64), 8-row groups together; `lead` is the step between 64-element column
// groups (only looked at where the contiguous axis is not the one summed over).
template <int ROW>
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(8 * ROW >> 4) << 32 | 1ull << 46 |
           (ROW == 128 ? 2ull : 4ull) << 61;
}
// f32 result, M = 128, operand types 0 (f16, or e4m3 of the 8-bit kind); bit 16: the second
// operand's contiguous axis is N
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool b_n_major) {
    return 1u << 4 | (b_n_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// Address of 16-byte chunk q (0-7) of row r within a 64-column half.
__device__ __forceinline__ uint32_t swz(uint32_t half, int r, int q) { return half + r * 128 + ((q ^ (r & 7)) << 4); }

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126..127

__device__ __forceinline__ bool is_dual(const Att& P, int mt) { return P.R - mt * 256 > 128; }

// The tiles of a CTA's segments, one after the other.
struct TileIter {
    SegIter it;
    Seg g;
    int seg, gt, t;                       // segment, tile of the CTA, tile of the item
    __device__ __forceinline__ void begin(const Att& P, const Stretch& st) {
        it.begin(P, st);
        seg = gt = -1;
        t = 0;
        g.t1 = 0;
    }
    __device__ __forceinline__ bool next(const Att& P) {
        ++gt;
        if (++t < g.t1) return true;
        if (!it.next(P, g)) return false;
        ++seg;
        t = g.t0;
        return true;
    }
    __device__ __forceinline__ bool cached() const { return t < g.q.nct; }
    __device__ __forceinline__ bool first() const { return t == g.t0; }
};

// This lane's page of a cached tile (lanes 0 to TILE / page - 1); -2: none.
__device__ __forceinline__ int page_entry(const Att& P, const Seg& g, int t, int lane) {
    const int ppt = TILE >> P.pshift, p = t * ppt + lane;
    return lane < ppt && p < g.q.full >> P.pshift ? __ldg(P.c.page_table + g.b * P.c.page_table_stride + p) : -2;
}

// The copying warp: the pages of a tile's keys, swizzled, then of its values, as they are.
template <int D>
__device__ void tc_copy_pages(const Att& P, const CUtensorMap* kmap, TcShared& sh, uint32_t base, const Stretch& st, int lane) {
    constexpr int KR = Tc<D>::KR, VR = Tc<D>::VR;
    TileIter u;
    u.begin(P, st);
    const uint32_t bytes = (uint32_t)D << P.pshift;
    int nk = 0, nv = 0, ahead = -2, ahead_t = -1, ahead_b = -1;
    unsigned k_sent = 0;                                  // of the units of keys before nk, bit 0 the last: whether a copy was sent
    // Whether no wait of the CTA has been given up.  This warp stops at the first: what it has sent are the last units then.
    auto wait = [&](uint64_t* b, uint32_t parity) {
        bar_wait(b, parity, sh);
        return __all_sync(FULL, !aborted(sh)) != 0;
    };
    bool ok = true;
    while (ok && u.next(P)) {
        // The tail does not lie in pages; it takes two units of keys, which this warp sees pass: a barrier's parity
        // says nothing to a waiter that is two phases behind or ahead.  So it also arrives at the units, which cannot be
        // used, and their barriers cannot go on, before it has.
        if (!u.cached()) {
            for (int i = 0; ok && i < 2; ++i) {
                ok = wait(&sh.ke[nk % KR], ((nk / KR) & 1) ^ 1);
                if (!ok) break;
                if (lane == 0) bar_arrive(&sh.kf[nk % KR]);
                k_sent <<= 1;
                ++nk;
            }
            continue;
        }
        const int page = ahead_b == u.g.b && ahead_t == u.t ? ahead : page_entry(P, u.g, u.t, lane);
        ahead = page_entry(P, u.g, u.t + 1, lane);        // on its way for the tile after
        ahead_b = u.g.b;
        ahead_t = u.t + 1;
        const bool there = page >= 0 && page < P.c.num_pages;
        if (page != -2 && !there) sh.bad_seg[u.seg & 7] = u.seg + 1;
        const uint32_t all = __popc(__ballot_sync(FULL, there)) * bytes;
        const int ks = nk % KR, vs = nv % VR;
        const int64_t ph = (int64_t)page * P.Hkv + u.g.h;
        ok = wait(&sh.ke[ks], ((nk / KR) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
            bar_arrive(&sh.kf[ks]);                       // in the place of the operand warps
            bar_expect(&sh.kf[ks], all);
        }
        __syncwarp();
        if (there) tensor_copy(base + Tc<D>::K + ks * Tc<D>::RAW_B + lane * bytes, kmap, (int)(ph << P.pshift), &sh.kf[ks]);
        k_sent = k_sent << 1 | 1u;
        ++nk;
        ok = wait(&sh.re[vs], ((nv / VR) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) bar_expect(&sh.rf[vs], all);
        __syncwarp();
        if (there) bulk_copy(base + Tc<D>::RAW + vs * Tc<D>::RAW_B + lane * bytes, static_cast<const char*>(P.c.v_pages) + ph * bytes,
                             bytes, &sh.rf[vs]);
        ++nv;
    }
    // also after a wait that gave up: no copy is in flight when the CTA ends
    bool landed = true;
    for (int i = nk - 1; i >= max(0, nk - KR); --i, k_sent >>= 1)
        if (k_sent & 1) landed &= bar_try(&sh.kf[i % KR], (i / KR) & 1) || bar_wait_slow(&sh.kf[i % KR], (i / KR) & 1, nullptr);
    for (int i = nv - 1; i >= max(0, nv - VR); --i)
        landed &= bar_try(&sh.rf[i % VR], (i / VR) & 1) || bar_wait_slow(&sh.rf[i % VR], (i / VR) & 1, nullptr);
    if (!landed) atomicOr(P.status, 1u << SPEC_ERR_COPY_IN_FLIGHT);
}

__device__ __forceinline__ void prefetch_row(const char* p, int bytes) {
    for (int i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" :: "l"(p + i));
}
// Rows that a segment's loads will ask for one after the other, on their way to L2 long before: its tail, and the
// queries of the segment after it.
template <int D>
__device__ void prefetch_segment(const Att& P, const TileIter& u, int lane) {
    const Seg& g = u.g;
    if (g.t1 > g.q.nct && g.q.len >= 0 && !g.q.bad) {
        const int64_t ring = ((int64_t)g.q.slot * P.Hkv + g.h) * 2 * P.page;
        for (int e = lane; e < g.q.open + P.N; e += 32) {
            const int64_t at = (ring + ((g.q.full + e) & (2 * P.page - 1))) * D * 2, n = e - g.q.open;
            prefetch_row(e < g.q.open ? static_cast<const char*>(P.c.k_open) + at : P.k.p + g.b * P.k.b + n * P.k.n + g.h * P.k.h, D * 2);
            prefetch_row(e < g.q.open ? static_cast<const char*>(P.c.v_open) + at : P.v.p + g.b * P.v.b + n * P.v.n + g.h * P.v.h, D * 2);
        }
    }
    SegIter it = u.it;
    Seg s;
    if (!it.next(P, s)) return;
    for (int r = s.mt * 256 + lane; r < min(P.R, s.mt * 256 + 256); r += 32) {
        const int n = r / P.G;
        prefetch_row(P.q.p + s.b * P.q.b + n * P.q.n + (s.h * P.G + r - n * P.G) * P.q.h, D * 2);
    }
}

// The warp that gathers the scales of the cached tiles' groups of 16 keys, a tile ahead.
template <int D>
__device__ __forceinline__ void tc_scales(const Att& P, TcShared& sh, const Stretch& st, int lane) {
    TileIter u;
    u.begin(P, st);
    auto fetch = [&](const Seg& g, int t, float& ks, float& vs) {
        ks = vs = 1.f;
        const int tok = t * TILE + lane * 16;
        if (lane < 8 && t < g.q.nct && tok < g.q.full) {
            const int id = __ldg(P.c.page_table + g.b * P.c.page_table_stride + (tok >> P.pshift));
            if (id >= 0 && id < P.c.num_pages) {
                ks = __ldg(P.c.k_scale + (int64_t)id * P.Hkv + g.h);
                vs = __ldg(P.c.v_scale + (int64_t)id * P.Hkv + g.h);
            }
        }
    };
    float ks = 1.f, vs = 1.f;
    bool more = u.next(P);
    if (more) {
        fetch(u.g, u.t, ks, vs);
        prefetch_segment<D>(P, u, lane);
    }
    while (more) {
        const int m = u.gt & (TC_META - 1);
        const uint32_t par = ((u.gt / TC_META) & 1) ^ 1;
        const bool cached = u.cached();
        const float k0 = ks, v0 = vs;
        more = u.next(P);
        if (more) fetch(u.g, u.t, ks, vs);
        if (more && u.first()) prefetch_segment<D>(P, u, lane);
        bar_wait(&sh.me[m], par, sh);
        // the operand warps write the tail's; they arrive once and this warp once (for the reason given at the copies)
        const bool far = __any_sync(FULL, is_far(v0));    // lanes without a key hold 1
        if (cached && lane < 8) {
            const float b = log2f(v0);
            sh.meta[m][0][lane] = k0;
            sh.meta[m][1][lane] = far ? -NEG_INF : b;
            sh.meta[m][2][lane] = far ? -1.f : 1.f / v0;
            if (far) sh.meta[m][3][lane] = b;
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&sh.mf[m]);
        if (lane == 0 && cached) bar_arrive(&sh.mf[m]);
    }
}

// Largest finite magnitude of bf16 words, as bits; elements that are not finite become 0 or (keep_nan) NaN.
template <int N>
__device__ __forceinline__ uint32_t bf16_amax(uint32_t (&w)[N], bool& bad, bool keep_nan) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    bad = m >= 0x7f80u;
    if (bad) {
        m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int s = 0; s < 32; s += 16) {
                const uint32_t a = (w[i] >> s) & 0x7fffu;
                if (a >= 0x7f80u) w[i] = (w[i] & ~(0xffffu << s)) | (keep_nan ? 0x7fffu << s : 0u);
                else m = max(m, a);
            }
    }
    return m;
}
__device__ __forceinline__ int bits_exp(uint32_t m) { return m ? max(min((int)(m >> 7), 253), 1) - 127 : 0; }

// The warps that make operands.
template <int D>
struct TcConv {
    static constexpr int CPR = D / 16;                    // 16-byte chunks of a cached row
    static constexpr int RPP = TC_CONV / CPR;             // rows per pass
    static constexpr int NP = TILE / RPP;                 // passes
    static constexpr int LPR = D / 8, RP = TC_CONV / LPR; // bf16 rows: lanes per row, rows per pass
    const Att& P;
    TcShared& sh;
    const uint32_t base;
    const int tid, lane;

    __device__ __forceinline__ TcConv(const Att& P_, TcShared& s, uint32_t b, int tid_)
        : P(P_), sh(s), base(b), tid(tid_), lane(tid_ & 31) {}

    __device__ __forceinline__ void arrive(uint64_t* bar) {
        proxy_fence();
        __syncwarp();
        if (lane == 0) bar_arrive(bar);
    }
    // A unit's bytes as f16 rows, rows from `valid` on as zeros.  The upper half of the lanes that share a row
    // stores its two chunks in the other order, so that eight lanes meet all 32 banks.
    __device__ __forceinline__ void put(uint32_t dst, uint32_t src, int valid) {
        const int c = tid % CPR, r0 = tid / CPR;
        const uint32_t half = dst + (c / 4) * Tc<D>::HALF;
        const int q = (c % 4) * 2, flip = c / 4;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int r = r0 + i * RPP;
            uint4 x = lds128(src + r * D + c * 16);
            if (r >= valid) x = make_uint4(0, 0, 0, 0);
            const uint2 a = e4m3_f16(x.x), b = e4m3_f16(x.y), d = e4m3_f16(x.z), e = e4m3_f16(x.w);
            const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(d.x, d.y, e.x, e.y);
            sts128(swz(half, r, q + flip), flip ? hi : lo);
            sts128(swz(half, r, q + 1 - flip), flip ? lo : hi);
        }
    }
    // Eight bf16 elements of a row in each of D / 8 lanes: the row's power of two, from the bits of its finite
    // magnitudes.  An element that is not finite is made 0 (a NaN with keep_nan) and reported.
    __device__ __forceinline__ int scale_row(uint4& w, bool& bad, bool keep_nan) {
        uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
        bad = (m & 0xffffu) >= 0x7f80u || m >= 0x7f800000u;
        if (bad) m = strip(w, keep_nan);
        m = max(m & 0xffffu, m >> 16);
#pragma unroll
        for (int o = D / 16; o; o >>= 1) m = max(m, __shfl_xor_sync(FULL, m, o));
        return m ? max((int)(m >> 7), 7) - 127 : 0;       // -120 to 127
    }
    static __device__ __noinline__ uint32_t strip(uint4& w, bool keep_nan) {
        uint32_t x[4] = {w.x, w.y, w.z, w.w}, m = 0;
        for (int i = 0; i < 4; ++i)
            for (int s = 0; s < 32; s += 16) {
                const uint32_t a = (x[i] >> s) & 0x7fffu;
                if (a >= 0x7f80u) x[i] = (x[i] & ~(0xffffu << s)) | (keep_nan ? 0x7fffu << s : 0u);
                else m = max(m, a);
            }
        w = make_uint4(x[0], x[1], x[2], x[3]);
        return m;
    }
    // The row times 2^e in f16: exact but for what lies below f16's smallest step.
    __device__ __forceinline__ void to_f16(const uint4& w, int e, uint32_t (&h)[4]) {
        const float s = exp2i(e);
        h[0] = pack_f16(bf_lo(w.x) * s, bf_hi(w.x) * s);
        h[1] = pack_f16(bf_lo(w.y) * s, bf_hi(w.y) * s);
        h[2] = pack_f16(bf_lo(w.z) * s, bf_hi(w.z) * s);
        h[3] = pack_f16(bf_lo(w.w) * s, bf_hi(w.w) * s);
    }
    // f16 value row r.
    __device__ __forceinline__ void put_value_row(uint32_t dst, int r, int l, const uint4& w, int e) {
        uint32_t h[4];
        to_f16(w, -e, h);
        sts128(swz(dst + (l / 8) * Tc<D>::HALF, r, l % 8),
               make_uint4(h[0], h[1], h[2], h[3]));
    }
    // The two e4m3 rows of a bf16 row divided by 2^(e - 7); the second's elements are exact differences.
    __device__ __forceinline__ void split_row(const uint4& w, int e, uint2& hi, uint2& lo) {
        uint32_t h[4], a[4], b[4];
        to_f16(w, 7 - e, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm("{\n\t.reg .b16 p, q;\n\t.reg .b32 f, d;\n\tcvt.rn.satfinite.e4m3x2.f16x2 p, %2;\n\tcvt.rn.f16x2.e4m3x2 f, p;\n\t"
                "sub.f16x2 d, %2, f;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, d;\n\tcvt.u32.u16 %0, p;\n\tcvt.u32.u16 %1, q;\n\t}"
                : "=r"(a[i]), "=r"(b[i]) : "r"(h[i]));
        }
        hi = make_uint2(a[0] | a[1] << 16, a[2] | a[3] << 16);
        lo = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
    }
    // The item's queries: QL lanes to a row, each with four (D = 64: two) pieces of 16 bytes, the next pass's on their way.
    // A loop that stays small: its code runs once per item and is never in the instruction caches.  (16 lanes to a row
    // and a piece each: 1100 cycles for 16 rows, nearly all of it waiting for shuffles.)
    static constexpr int QV = D / 32, QP = TC_CONV / 4;
    __device__ __forceinline__ void load_q(const Seg& g, int rows, int p, Bf16x8 (&w)[QV]) {
        const int r = min(tid / 4 + p * QP, rows - 1);    // rows behind the last repeat it
        const int row = g.mt * 256 + r, n = row / P.G, h = g.h * P.G + row - n * P.G;
        const char* src = P.q.p + g.b * P.q.b + n * P.q.n + h * P.q.h + 16 * (tid % 4);
#pragma unroll
        for (int i = 0; i < QV; ++i) w[i].load(src + 64 * i);
    }
    __device__ __forceinline__ void put_q_rows(Bf16x8 (&w)[QV], int p, float* rq) {
        const int r = tid / 4 + p * QP;
        uint32_t all[QV * 4];
#pragma unroll
        for (int i = 0; i < QV * 4; ++i) all[i] = (&w[i / 4].a.x)[i % 4];
        bool bad;
        uint32_t mx = bf16_amax(all, bad, true);
        mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
        const int e = mx ? max((int)(mx >> 7), 7) - 127 : 0;  // -120 to 127
        const uint32_t dst = base + Tc<D>::Q + (r / 128) * Tc<D>::Q_B;
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            const int l = tid % 4 + 4 * i;                // piece of the row
            uint2 hi, lo;
            split_row(make_uint4(all[4 * i], all[4 * i + 1], all[4 * i + 2], all[4 * i + 3]), e, hi, lo);
            // D = 128: two tiles of 128-byte rows; 64: side by side
            sts64(swz(dst, r % 128, l / 2) + (l & 1) * 8, hi);
            sts64((D == 128 ? swz(dst + Tc<D>::RAW_B, r % 128, l / 2) : swz(dst, r % 128, 4 + l / 2)) + (l & 1) * 8, lo);
        }
        if (tid % 4 == 0) rq[r] = exp2i(e) * (P.scale * 0.0078125f);
    }
    __device__ __forceinline__ void put_q(const Seg& g, int seg) {
        // the rows behind the last are whatever they are: their results are not looked at
        const int rows = min(256, P.R - g.mt * 256), np = (rows + QP - 1) / QP;
        float* rq = sh.rq[seg & 3];
        Bf16x8 w[QV];
        load_q(g, rows, 0, w);
#pragma unroll 1
        for (int p = 0; p < np; ++p) {
            Bf16x8 x[QV];
#pragma unroll
            for (int i = 0; i < QV; ++i) x[i] = w[i];
            load_q(g, rows, p + 1, w);                    // behind the last pass: the last row again
            put_q_rows(x, p, rq);
        }
    }
    // Row e of the tail: open tokens from the ring, then the nodes.  One load for every row, from a place that is
    // there (a query where there is no key): a branch per row would wait for each load in turn.
    __device__ __forceinline__ void load_tail(const TileIter& u, int p, Bf16x8& k, Bf16x8& v) {
        const int l = tid % LPR;
        const Seq& q = u.g.q;
        const int e = (u.t - q.nct) * TILE + tid / LPR + p * RP;
        const bool in = q.len >= 0 && !q.bad && e < q.open + P.N;
        const bool open = e < q.open;
        const int64_t at = ((((int64_t)q.slot * P.Hkv + u.g.h) * 2 * P.page + ((q.full + e) & (2 * P.page - 1))) * D) * 2;
        const int64_t n = e - q.open;
        const char* kp = open ? static_cast<const char*>(P.c.k_open) + at : P.k.p + u.g.b * P.k.b + n * P.k.n + u.g.h * P.k.h;
        const char* vp = open ? static_cast<const char*>(P.c.v_open) + at : P.v.p + u.g.b * P.v.b + n * P.v.n + u.g.h * P.v.h;
        k.load((in ? kp : P.q.p) + 16 * l);
        v.load((in ? vp : P.q.p) + 16 * l);
        if (!in) {
            k.zero();
            v.zero();
        }
    }
    __device__ __forceinline__ void put_tail_row(const TileIter& u, Bf16x8 k, Bf16x8 v, int p, uint32_t khi,
                                                 uint32_t klo, uint32_t vd, float* meta) {
        const int l = tid % LPR, r = tid / LPR + p * RP;
        bool bad;
        const int ve = min(scale_row(v.a, bad, false), 126);   // what is not finite reaches its rows at the end
        if (bad) {
            const int e = (u.t - u.g.q.nct) * TILE + r;
            atomicOr(&sh.bad_v[u.seg & 3][e >> 5], 1u << (e & 31));
        }
        put_value_row(vd, r, l, v.a, ve);
        const int ke = scale_row(k.a, bad, true);
        uint2 hi, lo;
        split_row(k.a, ke, hi, lo);
        sts64(key_at(khi, r, l), hi);
        sts64(key_at(klo, r, l), lo);
        if (l == 0) {
            meta[r] = exp2i(ke) * 0.0078125f;
            meta[TILE + r] = (float)ve;
            meta[2 * TILE + r] = exp2i(-ve);
            if (is_far_exp(ve)) *reinterpret_cast<volatile int*>(&sh.far_tail) = u.gt + 1;
        }
    }
    // A tile of the tail: its two units of keys, its values and all of its scales.
    __device__ __forceinline__ void tail(const TileIter& u, int nk) {
        constexpr int KR = Tc<D>::KR;
        const int m = u.gt & (TC_META - 1);
        const int k0 = nk % KR, k1 = (nk + 1) % KR;
        Bf16x8 ka{}, va{}, kb{}, vb{};
        bar_wait(&sh.me[m], ((u.gt / TC_META) & 1) ^ 1, sh);
        bar_wait(&sh.ke[k0], ((nk / KR) & 1) ^ 1, sh);
        bar_wait(&sh.ke[k1], (((nk + 1) / KR) & 1) ^ 1, sh);
        bar_wait(&sh.ve[u.gt & 1], ((u.gt >> 1) & 1) ^ 1, sh);
        const uint32_t khi = base + Tc<D>::K + k0 * Tc<D>::RAW_B, klo = base + Tc<D>::K + k1 * Tc<D>::RAW_B;
        const uint32_t vd = base + Tc<D>::V + (u.gt & 1) * Tc<D>::V_B;
        float* meta = sh.meta[m][0];
        // rows behind the last key: their scores are masked, their values have to be finite
        const int keys = u.g.q.len >= 0 && !u.g.q.bad ? min(TILE, u.g.q.open + P.N - (u.t - u.g.q.nct) * TILE) : 0;
        const int np = (keys + RP - 1) / RP;
        for (int i = np * RP * (D / 8) + tid; i < TILE * (D / 8); i += TC_CONV)
            sts128(swz(vd + (i % (D / 8) / 8) * Tc<D>::HALF, i / (D / 8), i % 8), make_uint4(0, 0, 0, 0));
        for (int r = np * RP + tid; r < TILE; r += TC_CONV) meta[r] = meta[TILE + r] = meta[2 * TILE + r] = 1.f;
#pragma unroll 1
        for (int p = -2; p < np; ++p) {
            const Bf16x8 k = ka, v = va;
            ka = kb;
            va = vb;
            load_tail(u, p + 2, kb, vb);
            if (p >= 0) put_tail_row(u, k, v, p, khi, klo, vd, meta);
        }
        proxy_fence();
        asm volatile("bar.sync 2, %0;" :: "n"(TC_CONV) : "memory");
        if (tid < 32 && *reinterpret_cast<volatile int*>(&sh.far_tail) == u.gt + 1) {
            for (int r = tid; r < TILE; r += 32) {
                meta[3 * TILE + r] = meta[TILE + r];
                meta[TILE + r] = -NEG_INF;
                meta[2 * TILE + r] = -1.f;
            }
            __syncwarp();
        }
        if (tid == 0) {
            bar_arrive(&sh.mf[m]);
            if (!aborted(sh)) {                           // else these units may not be free
                bar_arrive(&sh.kf[k0]);
                bar_arrive(&sh.kf[k1]);
            }
        }
        if (lane == 0) bar_arrive(&sh.vf[u.gt & 1]);
    }
    // Eight e4m3 of row r, as the tensor copy lays them: rows of D bytes, swizzled over D bytes.
    __device__ __forceinline__ uint32_t key_at(uint32_t dst, int r, int l) {
        const int q = D == 128 ? (l / 2) ^ (r & 7) : (l / 2) ^ ((r >> 1) & 3);
        return dst + r * D + q * 16 + (l & 1) * 8;
    }
    __device__ __forceinline__ void run(const Stretch& st) {
        constexpr int VR = Tc<D>::VR;
        TileIter u;
        u.begin(P, st);
        int nk = 0, nv = 0;
        while (u.next(P)) {
            if (u.first()) {
                bar_wait(&sh.qe, (u.seg & 1) ^ 1, sh);
                if (tid < 12) sh.bad_v[u.seg & 3][tid] = 0;
                asm volatile("bar.sync 2, %0;" :: "n"(TC_CONV) : "memory");
                put_q(u.g, u.seg);
                arrive(&sh.qf);
            }
            if (!u.cached()) {
                tail(u, nk);
                nk += 2;
                continue;
            }
            ++nk;
            const int s = nv % VR;
            bar_wait_copy(&sh.rf[s], (nv / VR) & 1, sh, P.wait_tries);
            bar_wait(&sh.ve[u.gt & 1], ((u.gt >> 1) & 1) ^ 1, sh);
            put(base + Tc<D>::V + (u.gt & 1) * Tc<D>::V_B, base + Tc<D>::RAW + s * Tc<D>::RAW_B, u.g.q.full - u.t * TILE);
            __syncwarp();
            if (lane == 0) bar_arrive(&sh.re[s]);
            ++nv;
            arrive(&sh.vf[u.gt & 1]);
        }
    }
};

// A row's bits of 32 of a tile's keys.
__device__ __forceinline__ uint32_t tile_mask(const Att& P, const Seg& g, int t, int n, int w) {
    if (t >= g.q.nct) return g.q.len < 0 || g.q.bad ? 0u : tail_bits(P, g.b, n, g.q.open, (t - g.q.nct) * TILE + 32 * w);
    const int left = g.q.full - t * TILE - 32 * w;
    return left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
}

// The column loops stay rolled: unrolled (and with the scores of 32 columns loaded ahead) the code no longer fits the
// instruction caches beside that of the other roles, and a round of 64-node trees took 800 us instead of 630.
__device__ __forceinline__ float group_max(const uint32_t (&r)[32], int u) {
    float a = __uint_as_float(r[16 * u]), b = __uint_as_float(r[16 * u + 1]);
#pragma unroll
    for (int j = 2; j < 14; j += 4) {
        a = max3(a, __uint_as_float(r[16 * u + j]), __uint_as_float(r[16 * u + j + 1]));
        b = max3(b, __uint_as_float(r[16 * u + j + 2]), __uint_as_float(r[16 * u + j + 3]));
    }
    a = max3(a, __uint_as_float(r[16 * u + 14]), __uint_as_float(r[16 * u + 15]));
    return fmaxf(a, b);
}
__device__ __forceinline__ float group_probs(const uint32_t (&r)[32], int u, float a, float b, uint32_t (&p)[16]) {
    float2 gs = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        float2 x = fma2(make_float2(__uint_as_float(r[16 * u + j]), __uint_as_float(r[16 * u + j + 1])), make_float2(a, a),
                        make_float2(b, b));
        x.x = ex2(x.x);
        x.y = ex2(x.y);
        gs = add2(gs, x);
        p[8 * u + j / 2] = pack_f16(x.x, x.y);
    }
    return gs.x + gs.y;
}
// A row's running maximum grows after `cols` of the tile's P have been written, four columns at a time: what has been summed so
// far (O, and these P) is brought to it.  Seldom taken once the first tiles are through.
template <int D>
__device__ __noinline__ void rescale(uint32_t s_col, uint32_t o_col, int cols, bool has_o, float f) {
    tc_wait_st();                        // the P that are read back
#pragma unroll 1
    for (int i = 0; i < cols; i += 4) {
        uint32_t p[4];
        tc_ld4(s_col + i, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {    // in f32: f may be too small for f16 where P f is not
            float x, y;
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(x), "=f"(y) : "r"(p[j]));
            p[j] = pack_f16(x * f, y * f);
        }
        tc_st4(s_col + i, p);
    }
    if (!has_o) return;
#pragma unroll 1
    for (int i = 0; i < D; i += 8) {
        uint32_t o[8];
        tc_ld8(o_col + i, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        tc_st8(o_col + i, o);
    }
}
constexpr float FAR_M = -3e38f;           // M of a far row, outside of this function
// Brings M up to mx where a row of the warp asks for it.
template <int D>
__device__ __forceinline__ void raise_m(uint32_t s_col, uint32_t o_col, int cols, bool has_o, float mx, float& m, float& l) {
    const float m2 = fmaxf(m, ceilf(mx)), f = m2 == NEG_INF ? 1.f : ex2(m - m2);
    m = m2;
    l *= f;
    if (cols > 0 || has_o) rescale<D>(s_col, o_col, cols, has_o, f);
}
// The rest of a tile, from column c on, for a warp whose rows are far: l is summed on its own, relative to 2^r.  What stands
// before column c weighs nothing (masked) or is NaN.  The thread's M, l and r are at x[0], x[2 TILE] and x[4 TILE] in shared memory.
template <int D>
__device__ __noinline__ void far_tile(uint32_t s_col, uint32_t o_col, int c, uint4 mk, int per, const float* meta, float rq, bool has_o,
                                      float* x) {
    float m = x[0], l = x[2 * TILE], r = x[4 * TILE];
    const float* b = meta + (meta[2 * TILE] < 0.f ? 3 * TILE : TILE);
#pragma unroll 1
    for (; c < TILE; c += 16) {
        const uint32_t bits = (c < 32 ? mk.x : c < 64 ? mk.y : c < 96 ? mk.z : mk.w) >> (c & 16);
        uint32_t v[16], p[8];
        tc_ld16(s_col + c, v);
        float mx = NEG_INF, top = NEG_INF, none = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float y = (bits >> j) & 1 ? __uint_as_float(v[j]) * fmaxf(meta[(c + j) >> per] * rq, 1.2e-38f) : NEG_INF;
            v[j] = __float_as_uint(y);
            top = fmaxf(top, y);
            mx = fmaxf(mx, y + b[(c + j) >> per]);
        }
        if (__any_sync(FULL, mx > m + M_SLACK)) raise_m<D>(s_col, o_col, c / 2, has_o, mx, m, none);
        if (top > r + R_SLACK) {
            const float up = ceilf(top);
            l *= moved(r, up);
            r = up;
        }
        const float sub = P_BIAS - (m == NEG_INF ? 0.f : m), ref = r == NEG_INF ? 0.f : r;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const float y = __uint_as_float(v[j]), z = __uint_as_float(v[j + 1]);
            l += ex2(y - ref) + ex2(z - ref);
            p[j / 2] = pack_f16(ex2(y + (b[(c + j) >> per] + sub)), ex2(z + (b[(c + j + 1) >> per] + sub)));
        }
        tc_st8(s_col + c / 2, p);
    }
    x[0] = m;
    x[2 * TILE] = l;
    x[4 * TILE] = r;
}
// Seldom taken once the first tiles are through: a row's largest w passes M + M_SLACK.  The weights of a far tile pass every M, and
// everything passes that of a far row: true then, and the tile from column c on has been dealt with.  So
// what is far costs the other rows nothing.
template <int D>
__device__ __forceinline__ bool grow(uint32_t s_col, uint32_t o_col, int c, const uint32_t (&mk)[4], int per, const float* meta, float rq,
                                     bool has_o, TcShared& sh, float mx, float& m, float& l) {
    if (!__any_sync(FULL, mx > m + M_SLACK)) return false;
    if (meta[2 * TILE] < 0.f || m == FAR_M) {             // the same for all rows of the warp
        float* const x = &sh.far[0][0][threadIdx.x];      // the softmax warps' threads are 0 to 255
        if (m != FAR_M) {
            x[0] = m;
            x[2 * TILE] = l;
            x[4 * TILE] = m == NEG_INF ? NEG_INF : m - P_BIAS;
            m = FAR_M;
        }
        far_tile<D>(s_col, o_col, c, make_uint4(mk[0], mk[1], mk[2], mk[3]), per, meta, rq, has_o, x);
        return true;
    }
    raise_m<D>(s_col, o_col, c / 2, has_o, mx, m, l);
    return false;
}

// A row of the streams joined where it is far in one of them: the factors of O, M, l, M - P_BIAS - r.
struct Joined {
    float f0, f1, m, l, lift;
};
__device__ __noinline__ Joined join_far(const TcShared& sh, int row, int nt) {
    float mi[2], li[2], ri[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool far = sh.xm[i][row] == FAR_M;
        mi[i] = far ? sh.far[0][i][row] : sh.xm[i][row];
        li[i] = far ? sh.far[1][i][row] : sh.xl[i][row];
        ri[i] = far ? sh.far[2][i][row] : mi[i] == NEG_INF ? NEG_INF : mi[i] - P_BIAS;
    }
    const float m = fmaxf(mi[0], mi[1]), r = fmaxf(ri[0], ri[1]);
    return Joined{moved(mi[0], m), nt < 2 ? 0.f : moved(mi[1], m), m,
                  li[0] * moved(ri[0], r) + (nt < 2 ? 0.f : li[1] * moved(ri[1], r)), lift_of(m, r)};
}

// One pass over a tile's scores: P = 2^(w - m + P_BIAS) in f16 over the scores, with m the largest w up to M_SLACK ago.
// A cached tile that has all of its keys, 32 at a time.
template <int D>
__device__ __forceinline__ void tile_softmax(uint32_t s_col, uint32_t o_col, const float* meta, float rq, bool has_o, TcShared& sh, float& m,
                                             float& l) {
    const uint32_t all[4] = {~0u, ~0u, ~0u, ~0u};
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t r[32], p[16];
        tc_ld32(s_col + 32 * c, r);
        tc_wait_ld(r);
        float mx = NEG_INF, a[2], b[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            a[u] = fmaxf(meta[2 * c + u] * rq, 1.2e-38f);
            b[u] = meta[TILE + 2 * c + u];
            mx = fmaxf(mx, fmaf(group_max(r, u), a[u], b[u]));
        }
        if (grow<D>(s_col, o_col, 32 * c, all, 4, meta, rq, has_o, sh, mx, m, l)) return;
        const float sub = P_BIAS - (m == NEG_INF ? 0.f : m);
#pragma unroll
        for (int u = 0; u < 2; ++u) l = fmaf(group_probs(r, u, a[u], b[u] + sub, p), meta[2 * TILE + 2 * c + u], l);
        tc_st16(s_col + 16 * c, p);      // columns that have been read
    }
}
// A masked one: the last of the cached tiles (a scale per 16 keys), and the tail (a scale per key).  Once or twice per item, so
// its instructions are never in the caches: it is kept small.
template <int D>
__device__ __forceinline__ void tile_softmax_masked(uint32_t s_col, uint32_t o_col, const uint32_t (&mk)[4], bool per_key,
                                                    const float* meta, float rq, bool has_o, TcShared& sh, float& m, float& l) {
    const int per = per_key ? 0 : 4;
    uint32_t bits = 0;
#pragma unroll 1
    for (int c = 0; c < TILE; c += 16, bits >>= 16) {
        if ((c & 16) == 0) bits = c == 0 ? mk[0] : c == 32 ? mk[1] : c == 64 ? mk[2] : mk[3];
        uint32_t r[16], p[8];
        tc_ld16(s_col + c, r);
        float mx = NEG_INF;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float* s = meta + ((c + j) >> per);
            const float x = fmaf(__uint_as_float(r[j]), fmaxf(s[0] * rq, 1.2e-38f), s[TILE]);
            r[j] = (bits >> j) & 1 ? __float_as_uint(x) : 0xff800000u;
            mx = fmaxf(mx, __uint_as_float(r[j]));
        }
        if (grow<D>(s_col, o_col, c, mk, per, meta, rq, has_o, sh, mx, m, l)) return;
        const float sub = P_BIAS - (m == NEG_INF ? 0.f : m);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const float x = ex2(__uint_as_float(r[j]) + sub), y = ex2(__uint_as_float(r[j + 1]) + sub);
            l = fmaf(x, meta[2 * TILE + ((c + j) >> per)], l);
            l = fmaf(y, meta[2 * TILE + ((c + j + 1) >> per)], l);
            p[j / 2] = pack_f16(x, y);
        }
        tc_st8(s_col + c / 2, p);
    }
}

// A partial result: the output rows, then the rows' M - P_BIAS, l and r; a multiple of 16 bytes.  r is only there where it is not
// M - P_BIAS, and l is negative then.
__host__ __device__ constexpr size_t partial_floats(size_t rows, int D) { return (rows * (D + 3) + 3) / 4 * 4; }
template <int D>
__device__ __forceinline__ float* partial_of(const Att& P, int cta, int slot) {
    return P.partial + ((int64_t)cta * 2 + slot) * partial_floats(min(P.R, 256), D);
}

__device__ __forceinline__ int rows_of(const Att& P) { return min(P.R, 256); }

template <int D>
__global__ void __launch_bounds__(TC_BT, 1) k_attention_tc(const Att P, const __grid_constant__ CUtensorMap kmap) {
    extern __shared__ unsigned char raw_smem[];
    const uint32_t base = (smem_u32(raw_smem) + 1023u) & ~1023u;
    TcShared& sh = *reinterpret_cast<TcShared*>(raw_smem + (base - smem_u32(raw_smem)) + Tc<D>::END);
    const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Stretch st = find_stretch<TC_BT>(P);
    if (tid == 0) P.cut[blockIdx.x].parts = 0;
    if (st.lo >= st.hi) return;
    if (tid == 0) {
        for (int i = 0; i < 6; ++i) {
            bar_init(&sh.kf[i], 2);
            bar_init(&sh.ke[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            bar_init(&sh.rf[i], 1);
            bar_init(&sh.re[i], TC_CONV / 32);
            bar_init(&sh.mf[i], 2);
            bar_init(&sh.me[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.vf[i], TC_CONV / 32);
            bar_init(&sh.ve[i], 1);
            bar_init(&sh.sf[i], 1);
            bar_init(&sh.pf[i], 128);
            bar_init(&sh.pv[i], 1);
        }
        for (int i = 0; i < 8; ++i) sh.bad_seg[i] = 0;
        bar_init(&sh.qf, TC_CONV / 32);
        bar_init(&sh.qe, 1);
        bar_init(&sh.drain, 1);
        sh.abort = sh.far_tail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        proxy_fence();
    }
    if (warp == TC_W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_before();
    }
    __syncthreads();
    tc_after();
    const uint32_t tmem = __shfl_sync(FULL, *reinterpret_cast<volatile uint32_t*>(&sh.tmem), 0);

    if (warp >= TC_W_CONV && warp < TC_W_MMA) {
        TcConv<D>(P, sh, base, tid - TC_SOFTMAX).run(st);
    } else if (warp == TC_W_COPY) {
        tc_copy_pages<D>(P, &kmap, sh, base, st, lane);
    } else if (warp == TC_W_SCALE) {
        tc_scales<D>(P, sh, st, lane);
    } else if (warp == TC_W_MMA) {
        // ---- matrix instructions
        const uint32_t lead = elect_one();
        SegIter it;
        Seg g;
        it.begin(P, st);
        uint32_t cnt[2] = {0, 0};
        int g0 = 0, nk0 = 0;
        constexpr uint32_t ID_QK = tc_idesc(TILE, false), ID_PV = tc_idesc(D, true);
        constexpr int KR = Tc<D>::KR;
        const uint64_t qd = tc_desc<128>(base + Tc<D>::Q, 16), kd = tc_desc<D>(base + Tc<D>::K, 16);
        const uint64_t vd = tc_desc<128>(base + Tc<D>::V, Tc<D>::HALF);
        for (int seg = 0; it.next(P, g); ++seg) {
            const bool dual = is_dual(P, g.mt);
            const int nt = g.t1 - g.t0, nc = max(0, min(nt, g.q.nct - g.t0));        // tiles, cached ones
            int left = dual ? 2 * nt : nt;                // score products still to issue
            bar_wait(&sh.qf, seg & 1, sh);
            tc_after();
            // Products of the two kinds are not ordered among themselves: a stream's probabilities have to be through
            // before its next scores are written over them.
            auto scores = [&](int i, int tl) {
                const uint32_t done = i ? cnt[1] : cnt[0];
                if (done) bar_wait(&sh.pv[i], (done - 1) & 1, sh);
                const uint64_t q = qd + (dual && i ? Tc<D>::Q_B >> 4 : 0);
                const int parts = tl < nc ? 1 : 2, nk = nk0 + tl + max(0, tl - nc);
                for (int part = 0; part < parts; ++part) {
                    const int s = (nk + part) % KR;
                    bar_wait_copy(&sh.kf[s], ((nk + part) / KR) & 1, sh, P.wait_tries);
                    tc_after();
                    const uint64_t k = kd + s * (Tc<D>::RAW_B >> 4);
#pragma unroll
                    for (int u = 0; u < 2 * D / 32; ++u) {         // q's first rows, then its second
                        const uint32_t off = D == 128 ? (u / 4) * Tc<D>::RAW_B + (u % 4) * 32 : u * 32;
                        tc_mma_e4m3(tmem + i * TILE, q + (off >> 4), k + (u % (D / 32)) * 2, ID_QK, part > 0 || u > 0, lead);
                    }
                    if (!dual || i == 1) tc_commit(&sh.ke[s], lead);
                }
                tc_commit(&sh.sf[i], lead);
                if (--left == 0) tc_commit(&sh.qe, lead);
            };
            auto tile = [&](int i, int step) { return dual ? step : 2 * step + i; };
#pragma unroll 1
            for (int i = 0; i < 2; ++i)
                if (tile(i, 0) < nt) scores(i, tile(i, 0));
#pragma unroll 1
            for (int n = 0; tile(0, n >> 1) < nt; ++n) {  // step n / 2 of stream n mod 2
                const int i = n & 1, step = n >> 1, tl = tile(i, step);
                if (tl >= nt) continue;
                const int gt = g0 + tl, s = gt & 1;
                const uint32_t done = i ? cnt[1] : cnt[0];
                bar_wait(&sh.vf[s], (gt >> 1) & 1, sh);
                bar_wait(&sh.pf[i], done & 1, sh);
                tc_after();
                const uint64_t v = vd + s * (Tc<D>::V_B >> 4);
#pragma unroll
                for (int u = 0; u < TILE / 16; ++u)
                    tc_mma_ts(tmem + Tc<D>::O_COL + i * D, tmem + i * TILE + u * 8, v + u * 128, ID_PV, step > 0 || u > 0, lead);
                cnt[0] += i == 0;
                cnt[1] += i == 1;
                if (!dual || i == 1) {
                    tc_commit(&sh.ve[s], lead);
                    tc_commit(&sh.me[gt & (TC_META - 1)], lead);
                }
                tc_commit(&sh.pv[i], lead);
                if (tile(i, step + 1) < nt) scores(i, tile(i, step + 1));
            }
            g0 += nt;
            nk0 += nt + (nt - nc);
        }
        tc_commit(&sh.drain, lead);
        // also after a wait that gave up: nothing runs on when the tensor memory is freed
        if (!bar_try(&sh.drain, 0)) bar_wait_slow(&sh.drain, 0, nullptr);
        __syncwarp();
    } else if (warp < TC_SOFTMAX / 32) {
        // ---- softmax of stream i; thread = row
        const int i = warp / 4, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;               // 32 lanes per warp, lane index in bits 16-31
        const uint32_t s_col = tmem + lanes + i * TILE, o_col = tmem + lanes + Tc<D>::O_COL;
        SegIter it;
        Seg g;
        it.begin(P, st);
        uint32_t cnt = 0;
        int g0 = 0;
        for (int seg = 0; it.next(P, g); ++seg) {
            const int rows = min(256, P.R - g.mt * 256);
            const bool dual = rows > 128;
            const int nt = g.t1 - g.t0;
            const int ri = dual ? i * 128 + r : r;                        // row of the item
            const int row = g.mt * 256 + min(ri, rows - 1), n = row / P.G, head = g.h * P.G + row % P.G;
            float m = NEG_INF, l = 0.f, rq = 0.f;
            bool any = false;
            const bool idle = ri - lane >= rows;
            for (int tl = dual ? 0 : i; tl < nt; tl += dual ? 1 : 2) {
                const int gt = g0 + tl, t = g.t0 + tl;
                const float* meta = sh.meta[gt & (TC_META - 1)][0];
                const bool masked = t >= g.q.nct || (t + 1) * TILE > g.q.full;
                uint32_t mk[4] = {};
                if (masked && !idle) {                                    // while the scores are made
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t bits = tile_mask(P, g, t, n, w);
                        mk[0] = w == 0 ? bits : mk[0];
                        mk[1] = w == 1 ? bits : mk[1];
                        mk[2] = w == 2 ? bits : mk[2];
                        mk[3] = w == 3 ? bits : mk[3];
                    }
                }
                bar_wait(&sh.sf[i], cnt & 1, sh);          // first: with it, the scales' barrier is in this phase or the next
                bar_wait(&sh.mf[gt & (TC_META - 1)], (gt / TC_META) & 1, sh);
                tc_after();
                const bool begins = !any;
                if (begins) rq = sh.rq[seg & 3][ri];
                any = true;
                ++cnt;
                if (idle) {                                               // no row in this warp: whatever P holds stays in its rows
                    tc_before();
                    bar_arrive(&sh.pf[i]);
                    continue;
                }
                // with this tile's scores the product before them has ended: O can be rescaled
                if (!masked) tile_softmax<D>(s_col, o_col + i * D, meta, rq, !begins, sh, m, l);
                else tile_softmax_masked<D>(s_col, o_col + i * D, mk, t >= g.q.nct, meta, rq, !begins, sh, m, l);
                tc_wait_st();
                tc_before();
                bar_arrive(&sh.pf[i]);
            }
            if (any) {
                bar_wait(&sh.pv[i], (cnt - 1) & 1, sh);
                tc_after();
            }
            // ---- the segment's rows: whole items are written out, parts go to the workspace
            float f[2] = {1.f, 0.f};                                      // factors of the streams' sums
            int c_lo = 0, c_hi = D;
            float lift = 0.f;                                             // M - P_BIAS - r
            if (!dual) {
                sh.xm[i][r] = m;
                sh.xl[i][r] = l;
                tc_before();
                asm volatile("bar.sync 1, %0;" :: "n"(TC_SOFTMAX) : "memory");
                tc_after();
                const float m0 = sh.xm[0][r], m1 = sh.xm[1][r], mm = fmaxf(m0, m1);
                f[0] = m0 == NEG_INF ? (mm == NEG_INF ? 1.f : 0.f) : ex2(m0 - mm);
                f[1] = nt < 2 ? 0.f : m1 == NEG_INF ? (mm == NEG_INF ? 1.f : 0.f) : ex2(m1 - mm);
                l = sh.xl[0][r] * f[0] + (nt < 2 ? 0.f : sh.xl[1][r] * f[1]);
                m = mm;
                if (m0 == FAR_M || m1 == FAR_M) {
                    const Joined j = join_far(sh, r, nt);
                    f[0] = j.f0, f[1] = j.f1, m = j.m, l = j.l, lift = j.lift;
                }
                c_lo = i * (D / 2);
                c_hi = c_lo + D / 2;
            } else if (m == FAR_M) {
                m = sh.far[0][i][r];
                l = sh.far[1][i][r];
                lift = lift_of(m, sh.far[2][i][r]);
            }
            const bool whole = g.whole();
            const bool invalid = g.q.bad || *reinterpret_cast<volatile int*>(&sh.bad_seg[seg & 7]) == seg + 1;
            if (invalid && r == 0) atomicOr(P.status, 1u << SPEC_ERR_DEVICE_INPUT);
            const bool nan = invalid || aborted(sh);
            uint32_t bad_v = 0;
            if (g.t1 > g.q.nct && !nan) {
#pragma unroll
                for (int w = 0; w < 12; ++w) bad_v |= sh.bad_v[seg & 3][w];
            }
            const float inv = (l == 0.f ? 0.f : 1.f / l) * (lift == 0.f ? 1.f : half_exp2(lift));
            const int64_t orow = ((int64_t)g.b * P.N + n) * P.Hq + head;
            float* part = partial_of<D>(P, blockIdx.x, g.t0 == 0 ? 1 : 0);
            const float quiet = __int_as_float(0x7fffffff);
#pragma unroll 1
            for (int c = c_lo; c < (idle ? c_lo : c_hi); c += 8) {
                uint32_t o[8];
                tc_ld8(o_col + (dual ? i * D : 0) + c, o);
                if (!dual) {
                    if (nt > 1) {
                        uint32_t o2[8];
                        tc_ld8(o_col + D + c, o2);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * f[0] + __uint_as_float(o2[j]) * f[1]);
                    }
                }
                if (bad_v) {                                              // values that could not enter the product
                    for (int w = 0; w < 12; ++w) {
                        uint32_t hit = sh.bad_v[seg & 3][w];
                        if (hit) hit &= tail_bits(P, g.b, n, g.q.open, 32 * w);
                        for (; hit; hit &= hit - 1) {
                            const int e = 32 * w + __ffs(hit) - 1;
                            const char* src = e < g.q.open
                                ? static_cast<const char*>(P.c.v_open) +
                                      (((int64_t)g.q.slot * P.Hkv + g.h) * 2 * P.page + (g.q.full + e) % (2 * P.page)) * D * 2
                                : P.v.p + g.b * P.v.b + (e - g.q.open) * P.v.n + g.h * P.v.h;
                            const __nv_bfloat16* vv = reinterpret_cast<const __nv_bfloat16*>(src) + c;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float x = __bfloat162float(vv[j]);
                                if (!(fabsf(x) <= 3.402823466e38f)) o[j] = __float_as_uint(__uint_as_float(o[j]) + x);
                            }
                        }
                    }
                }
                if (ri < rows) {
                    if (whole) {
                        uint32_t w[4];
                        if (lift != 0.f) {
                            const float up = half_exp2(lift);
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * up);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = nan ? 0x7fff7fffu : pack_bf16(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                        *reinterpret_cast<uint4*>(P.out + (orow * D + c) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        float4* dst = reinterpret_cast<float4*>(part + (int64_t)ri * D + c);
#pragma unroll
                        for (int j = 0; j < 8; j += 4)
                            dst[j / 4] = nan ? make_float4(quiet, quiet, quiet, quiet)
                                             : make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]),
                                                           __uint_as_float(o[j + 2]), __uint_as_float(o[j + 3]));
                    }
                }
            }
            const bool speaks = ri < rows && (dual || i == 0);
            if (whole) {
                if (speaks && P.lse) P.lse[orow] = nan ? quiet : l == 0.f ? NEG_INF : (m - P_BIAS - lift + log2f(l)) * LN2;
            } else {
                if (speaks) {
                    float* stat = part + (int64_t)rows_of(P) * D + ri;
                    stat[0] = m == NEG_INF ? NEG_INF : m - P_BIAS;
                    stat[rows_of(P)] = nan ? quiet : lift == 0.f ? l : -l;
                    if (lift != 0.f) stat[2 * rows_of(P)] = m - P_BIAS - lift;
                }
                if (g.t0 == 0 && tid == 0) P.cut[blockIdx.x] = Cut{g.b, g.h, g.mt, parts_of(P, g, st, blockIdx.x)};
            }
            // the next segment's products may write O again once every reader is through
            tc_before();
            if (!dual) asm volatile("bar.sync 1, %0;" :: "n"(TC_SOFTMAX) : "memory");
            g0 += nt;
        }
    }
    __syncthreads();
    if (warp == TC_W_MMA) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem));
        if (lane == 0 && sh.abort) atomicOr(P.status, 1u << SPEC_ERR_TIMEOUT);
    }
}

// Puts the cut items together: block x the item that CTA x began, one warp per
// row, lane p the references and the sum of part p.  Bound by latency: the parts lie in L2.
// Launched beside the kernel before, so that only its own work is left when that ends.  A row to each warp: with 4, 2, 1 of them
// one tree of 32 over 131072 tokens (8 items in 148 parts) took 126, 116, 111 us, 64 chains of 6 205, 200, 197.
constexpr int MERGE_BT = 256, MERGE_ROWS = MERGE_BT / 32;

template <int D>
__global__ void __launch_bounds__(MERGE_BT) k_attention_merge(const Att P) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Cut cut = P.cut[blockIdx.x];
    const int lane = threadIdx.x & 31, rows = rows_of(P);
    const int upto = min(min(rows, P.R - cut.mt * 256), (int)(blockIdx.y + 1) * MERGE_ROWS);
    if (cut.parts == 0) return;
    constexpr int E = D / 32;
    for (int r = blockIdx.y * MERGE_ROWS + (threadIdx.x >> 5); r < upto; r += MERGE_BT / 32) {
        auto part = [&](int i) { return partial_of<D>(P, blockIdx.x + i, i == 0 ? 1 : 0); };
        float M = NEG_INF, R = NEG_INF, m0 = NEG_INF, r0 = NEG_INF, l0 = 0.f;
        for (int i = lane; i < cut.parts; i += 32) {
            const float* p = part(i) + (int64_t)rows * D + r;
            const float m = __ldcg(p), s = __ldcg(p + rows), x = s < 0.f ? __ldcg(p + 2 * rows) : m;
            if (i == lane) m0 = m, l0 = s < 0.f ? -s : s, r0 = x;
            M = fmaxf(M, m);
            R = fmaxf(R, x);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
            R = fmaxf(R, __shfl_xor_sync(FULL, R, o));
        }
        const float base = M == NEG_INF ? 0.f : M, ref = R == NEG_INF ? 0.f : R;
        float acc[E] = {}, l = 0.f;
        for (int i0 = 0; i0 < cut.parts; i0 += 32) {
            if (i0) {
                m0 = r0 = NEG_INF, l0 = 0.f;
                if (i0 + lane < cut.parts) {
                    const float* p = part(i0 + lane) + (int64_t)rows * D + r;
                    m0 = r0 = __ldcg(p);
                    l0 = __ldcg(p + rows);
                    if (l0 < 0.f) l0 = -l0, r0 = __ldcg(p + 2 * rows);
                }
            }
            const float w = ex2(m0 - base);
            l = fmaf(ex2(r0 - ref), l0, l);
            const int n = min(32, cut.parts - i0);
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float wi = __shfl_sync(FULL, w, i);
                const float* p = part(i0 + i) + (int64_t)r * D + lane * E;
                if constexpr (E == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
                    acc[0] = fmaf(wi, x.x, acc[0]); acc[1] = fmaf(wi, x.y, acc[1]);
                    acc[2] = fmaf(wi, x.z, acc[2]); acc[3] = fmaf(wi, x.w, acc[3]);
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(p));
                    acc[0] = fmaf(wi, x.x, acc[0]); acc[1] = fmaf(wi, x.y, acc[1]);
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(FULL, l, o);
        const float up = half_exp2(M == NEG_INF ? 0.f : M - ref), inv = (l == 0.f ? 0.f : 1.f / l) * up;
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] = acc[j] * up * inv;
        const int row = cut.mt * 256 + r, n = row / P.G;
        const int64_t at = ((int64_t)cut.b * P.N + n) * P.Hq + cut.h * P.G + row - n * P.G;
        char* out = P.out + at * D * 2;
        if constexpr (E == 4)
            reinterpret_cast<uint2*>(out)[lane] = make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
        else
            reinterpret_cast<uint32_t*>(out)[lane] = pack_bf16(acc[0], acc[1]);
        if (P.lse && lane == 0) P.lse[at] = l == 0.f ? NEG_INF : (ref + log2f(l)) * LN2;
    }
}

// ----------------------------------------------------------------------------- few rows (mma.sync)

// At most 16 rows of a kv head (single tokens, short chains): bound by the bytes
// of the cache.  A warp takes 32 keys of each tile (two chunks of 16); tensor
// copies bring their bytes to a ring of two tiles in shared memory that is the warp's own, so
// that the next tile's are on their way while one is computed (8 KB for each of 12 warps at D = 128).
// From there they go straight into the fragments of m16n8k16 products, with the
// keys (scores) and the dims (output) as rows and 8 queries as columns: NQ = 1 for up
// to 8 rows of a kv head, 2 for up to 16.  The dimensions that are summed over, and the rows of the
// output, may stand in any order as long as both sides agree, so each lane reads 16 bytes where it
// needs them (the swizzle keeps the lanes on different banks).
//   scores  rows: lane (g, c) holds, of keys g and g + 8, the bytes [c D/4, (c + 1) D/4);
//           four of them feed one 16-wide step.  Columns: queries.
//   output  lane (g, c) holds, of keys 2c, 2c + 1, 2c + 8, 2c + 9, the dims [g D/8, (g + 1) D/8):
//           bytes 2t and 2t + 1 of two keys make the pairs that row block t wants in its rows g and g + 8.
// Probabilities leave the first product with a key per row and enter the second with a query per column:
// 8 x 8 transposes between registers.
// Each warp has its own running maximum, sum and output (in registers); the four
// are joined through shared memory at the end of an item.
//
// Measured (D = 128, 32 query on 8 kv heads): 64 single tokens over ragged lengths up to 8192 125 us, 5.4 TB/s, 0.83 of the copy
// rate.  Bound by the bytes, near the end by latency: three warps per scheduler issue in 37% of the cycles.  With queries as
// rows (16, half of them empty for 8) it took 140 us, with steps of 16 keys 170.
// Up to 16 rows go this way; the tensor-core kernel takes 128 rows in the time of one.  64 chains of 2 with 64 query heads,
// 16 rows, over 4096: 99 us here.  More rows
// by more warps on the same ring (queries as rows) were measured against it: 32 rows 223 : 211 us, 48 rows 226 : 219, 64 rows
// 320 : 229.
constexpr int MM_BT = 128, MM_WARPS = MM_BT / 32, MM_ROWS = 16, MM_CTAS_SM = 3;

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16_f16(uint32_t w, float s) { return pack_f16(bf_lo(w) * s, bf_hi(w) * s); }

// A warp's part of a tile.
struct Part {
    int tok, is;                          // the tile's first key; what it is, kv head, segment's parity
    __device__ __forceinline__ int kind() const { return is & 3; }       // 0 none left, 1 cached, 2 tail, 3 nothing to do
    __device__ __forceinline__ int h() const { return is >> 2 & 0xfff; }
    __device__ __forceinline__ int parity() const { return is >> 14; }
};
struct MmAhead {
    SegIter it;
    Seg s;
    int more;
};

// A warp's ring: two tiles' 2 x 16 keys and values; their pages' scales.
template <int D> struct MmRing {
    unsigned char k[2][2][16 * D], v[2][2][16 * D];
};
struct MmSlots {
    float scale[2][2][2];                                 // [slot][chunk][keys, values]
    float ref[16];                                        // r of the rows: once they are far, and at a segment's end
    uint64_t full[2];
};

template <int D, int NQ>
struct MmWarp {
    static constexpr int KH = D / 64;                     // 16-byte pieces of a key per lane
    static constexpr int VW = D / 32;                     // 4-byte words of a value per lane
    static constexpr int NT = D / 16;                     // row blocks of the output
    const Att& P;
    const int lane, warp, g, c;
    MmAhead& a;                                           // the segment of the chunk after, kept by lane 0
    float* const ref;                                     // r of the rows, in shared memory
    int t, parity;
    bool far;                                             // l is relative to 2^r, not to 2^(m - P_BIAS)
    // [column block][..]: dims g D/8 + 2t (0, 1) and + 1 (2, 3) of queries 2c and 2c + 1; their maxima and this lane's sums
    float o[NQ][NT][4], m[NQ][2], l[NQ][2];

    __device__ __forceinline__ MmWarp(const Att& P_, int warp_, MmAhead& a_, MmSlots& slots)
        : P(P_), lane(threadIdx.x & 31), warp(warp_), g(lane >> 2), c(lane & 3), a(a_), ref(slots.ref) {}

    __device__ __forceinline__ void begin(const Stretch& st) {
        if (lane == 0) {
            a.it.begin(P, st);
            a.s.t1 = 0;
        }
        __syncwarp();
        parity = 1;
        t = 0;
    }
    // The warp's part of the tile after, and in lanes 0 and 1 the pages of its two chunks (-2: none).
    __device__ __forceinline__ Part next(int& page) {
        Part x{};
        page = -2;
        if (++t >= a.s.t1) {
            __syncwarp();
            if (lane == 0) a.more = a.it.next(P, a.s);
            __syncwarp();
            if (!a.more) return x;
            parity ^= 1;
            t = a.s.t0;
        }
        const Seg& s = a.s;
        const bool cached = t < s.q.nct;
        x.tok = (cached ? t : t - s.q.nct) * TILE;
        x.is = (cached ? 1 : s.q.len >= 0 && !s.q.bad ? 2 : 3) | s.h << 2 | parity << 14;
        const int tok = x.tok + first_key(lane);
        if (cached && lane < 2 && tok < s.q.full) page = __ldg(P.c.page_table + s.b * P.c.page_table_stride + (tok >> P.pshift));
        return x;
    }
    __device__ __forceinline__ int first_key(int chunk) const { return 16 * (warp + MM_WARPS * chunk); }
    // A cached part's bytes and scales on their way to slot s of the ring: chunk h by lane h.  A chunk behind the last key,
    // or of a page that is not there, brings nothing.
    __device__ __forceinline__ void fetch(const Part& x, int id, int s, MmRing<D>& ring, MmSlots& slots, const CUtensorMap* kmap,
                                          const CUtensorMap* vmap) const {
        if (x.kind() != 1) return;
        __syncwarp();                                     // the slot has been read
        if (lane < 2) {
            if (id >= 0 && id < P.c.num_pages) {
                const int64_t ph = (int64_t)id * P.Hkv + x.h();
                const int row = (int)((ph << P.pshift) + ((x.tok + first_key(lane)) & (P.page - 1)));
                copy4(&slots.scale[s][lane][0], P.c.k_scale + ph);
                copy4(&slots.scale[s][lane][1], P.c.v_scale + ph);
                bar_expect(&slots.full[s], 2 * 16 * D);
                tensor_copy(smem_u32(ring.k[s][lane]), kmap, row, &slots.full[s]);
                tensor_copy(smem_u32(ring.v[s][lane]), vmap, row, &slots.full[s]);
            } else {
                bar_arrive(&slots.full[s]);
            }
            copy4_arrive(&slots.full[s]);
        }
    }
    __device__ __forceinline__ float own_ref(int q, int e) const { return m[q][e] == NEG_INF ? NEG_INF : m[q][e] - P_BIAS; }
    // From now on the segment's sums are far.
    __device__ __forceinline__ void go_far() {
        far = true;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (g == 0) ref[8 * q + 2 * c + e] = own_ref(q, e);
        __syncwarp();
    }
    // A far row's sum over NC x 16 keys, relative to 2^r.
    template <int NC, bool EACH>
    __device__ __forceinline__ void far_sums(const float (&s)[NC][NQ][4], const float (&rq)[NQ][2], const float (&a)[NC][2],
                                             const uint32_t (&mask)[NQ][2]) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x[2 * NC], top = NEG_INF;
#pragma unroll
                for (int n = 0; n < 2 * NC; ++n) {
                    x[n] = s[n >> 1][q][2 * (n & 1) + e] * fmaxf(a[n >> 1][n & 1] * rq[q][e], 1.2e-38f);
                    if (EACH && !((mask[q][e] >> (g + 8 * (n & 1))) & 1)) x[n] = NEG_INF;
                    top = fmaxf(top, x[n]);
                }
#pragma unroll
                for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
                float& at = ref[8 * q + 2 * c + e];       // the same row in all lanes of column c
                float r = at;
                __syncwarp();
                if (top > r + R_SLACK) {
                    const float up = ceilf(top);
                    l[q][e] *= moved(r, up);
                    r = up;
                    if (g == 0) at = r;
                }
                __syncwarp();
                const float sub = r == NEG_INF ? 0.f : r;
#pragma unroll
                for (int n = 0; n < 2 * NC; ++n) l[q][e] += ex2(x[n] - sub);
            }
    }
    // Scores of NC x 16 keys to probabilities (the second product's columns).  Of keys g (0) and g + 8 (1) of each chunk: a the
    // scale (the queries' factors rq come on top), b log2 of the value's, inv 1 / that.  EACH: these differ from key to key,
    // and mask bit 8 i says whether the query sees key g + 8 i.
    template <int NC, bool EACH>
    __device__ __forceinline__ void softmax(float (&s)[NC][NQ][4], const float (&rq)[NQ][2], const float (&a)[NC][2], const float (&b)[NC][2],
                                            const float (&inv)[NC][2], const uint32_t (&mask)[NQ][2], uint32_t (&p)[NC][NQ][2]) {
        bool grow = false;
        float top[NQ][2];
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = NEG_INF;
#pragma unroll
                for (int n = 0; n < NC; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float& x = s[n][q][2 * i + e];
                        x = fmaf(x, fmaxf(a[n][i] * rq[q][e], 1.2e-38f), b[n][i]);
                        if (EACH && !((mask[q][e] >> (g + 8 * i)) & 1)) x = NEG_INF;
                        mx = fmaxf(mx, x);
                    }
                top[q][e] = mx;
                grow |= mx > m[q][e] + M_SLACK;
            }
        if (__any_sync(FULL, grow)) {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(m[q][e], top[q][e]);
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, d));
                    const float f = mx == NEG_INF ? 1.f : ex2(m[q][e] - mx);
                    m[q][e] = mx;
                    if (!far) l[q][e] *= f;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        o[q][j][e] *= f;
                        o[q][j][2 + e] *= f;
                    }
                }
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            float sub[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) sub[e] = P_BIAS - (m[q][e] == NEG_INF ? 0.f : m[q][e]);
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float x = ex2(s[n][q][2 * i] + sub[0]), y = ex2(s[n][q][2 * i + 1] + sub[1]);
                    l[q][0] = fmaf(x, inv[n][i], l[q][0]);
                    l[q][1] = fmaf(y, inv[n][i], l[q][1]);
                    p[n][q][i] = transpose8(pack_f16(x, y));
                }
        }
    }
    // 16-byte piece q of row r of a slot, as the tensor copy swizzles it.
    static __device__ __forceinline__ uint32_t piece(uint32_t at, int r, int q) {
        return at + r * D + ((D == 128 ? q ^ (r & 7) : q ^ (r >> 1 & 3)) << 4);
    }
    // The queries of 16 dims: fragments of NQ columns.
    static __device__ __forceinline__ void columns(const uint32_t* qf, int u, int lane, uint32_t (&b)[NQ][2]) {
        if constexpr (NQ == 1) {
            const uint2 x = reinterpret_cast<const uint2*>(qf)[u * 32 + lane];
            b[0][0] = x.x; b[0][1] = x.y;
        } else {
            const uint4 x = reinterpret_cast<const uint4*>(qf)[u * 32 + lane];
            b[0][0] = x.x; b[0][1] = x.y; b[1][0] = x.z; b[1][1] = x.w;
        }
    }
    // The first NC chunks of a slot.
    template <int NC>
    __device__ __forceinline__ void cached(const MmRing<D>& ring, const MmSlots& slots, int sl, const uint32_t* qf, const float (&rq)[NQ][2]) {
        float s[NC][NQ][4] = {};
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            uint4 k[2 * NC];
#pragma unroll
            for (int i = 0; i < 2 * NC; ++i) k[i] = lds128(piece(smem_u32(ring.k[sl][i >> 1]), g + 8 * (i & 1), KH * c + j));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t b[NQ][2];
                columns(qf, j * 4 + u, lane, b);
#pragma unroll
                for (int n = 0; n < NC; ++n) {
                    const uint4 &k0 = k[2 * n], &k1 = k[2 * n + 1];
                    const uint2 x = e4m3_f16(u == 0 ? k0.x : u == 1 ? k0.y : u == 2 ? k0.z : k0.w);
                    const uint2 y = e4m3_f16(u == 0 ? k1.x : u == 1 ? k1.y : u == 2 ? k1.z : k1.w);
#pragma unroll
                    for (int q = 0; q < NQ; ++q) mma16816(s[n][q], x.x, y.x, x.y, y.y, b[q][0], b[q][1]);
                }
            }
        }
        float aa[NC][2], bb[NC][2], ii[NC][2];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const float vs = slots.scale[sl][n][1];
            aa[n][0] = aa[n][1] = slots.scale[sl][n][0];
            bb[n][0] = bb[n][1] = __log2f(vs);
            ii[n][0] = ii[n][1] = __frcp_rn(vs);
        }
        const uint32_t none[NQ][2] = {};
        uint32_t p[NC][NQ][2];
        bool wide = far;
#pragma unroll
        for (int n = 0; n < NC; ++n) wide |= is_far(slots.scale[sl][n][1]);
        if (wide) {                                       // the same in all lanes
            if (!far) go_far();
            far_sums<NC, false>(s, rq, aa, none);
#pragma unroll
            for (int n = 0; n < NC; ++n) ii[n][0] = ii[n][1] = 0.f;
        }
        softmax<NC, false>(s, rq, aa, bb, ii, none, p);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            uint32_t v[4][VW];
            const uint32_t vp = smem_u32(ring.v[sl][n]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 2 * c + (i & 1) + (i >> 1) * 8;
                if constexpr (VW == 4) {
                    const uint4 w = lds128(piece(vp, r, g));
                    v[i][0] = w.x; v[i][1] = w.y; v[i][2] = w.z; v[i][3] = w.w;
                } else {
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[i][0]), "=r"(v[i][1]) : "r"(piece(vp, r, g >> 1) + (g & 1) * 8));
                }
            }
#pragma unroll
            for (int u = 0; u < VW; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {             // bytes 2h, 2h + 1 of word u, of two keys side by side
                    const uint2 x = e4m3_f16(__byte_perm(v[0][u], v[1][u], h ? 0x7362 : 0x5140));
                    const uint2 y = e4m3_f16(__byte_perm(v[2][u], v[3][u], h ? 0x7362 : 0x5140));
#pragma unroll
                    for (int q = 0; q < NQ; ++q) mma16816(o[q][2 * u + h], x.x, x.y, y.x, y.y, p[n][q][0], p[n][q][1]);
                }
        }
    }
    // 16 keys of the tail, from bf16 rows.  bad_v: the item's keys whose value is not finite.
    __device__ __forceinline__ void tail(int tok, const Seg& sg, const uint32_t* qf, const float (&rq)[NQ][2], uint32_t* bad_v) {
        const Seq& q = sg.q;
        const int64_t ring = ((int64_t)q.slot * P.Hkv + sg.h) * 2 * P.page;
        auto row = [&](int e, int which) -> const char* {                // a place that is there for every row
            const int64_t at = (ring + ((q.full + e) & (2 * P.page - 1))) * D * 2, n = e - q.open;
            const sv_host::Rows& src = which ? P.v : P.k;
            const char* p = e < q.open ? static_cast<const char*>(which ? P.c.v_open : P.c.k_open) + at
                                       : src.p + sg.b * src.b + n * src.n + sg.h * src.h;
            return e < q.open + P.N ? p : P.q.p;
        };
        const int keys = q.open + P.N;
        float s[1][NQ][4] = {}, aa[1][2], bb[1][2], ii[1][2], ks[2];
        uint32_t kw[2][KH * 8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const char* p = row(tok + 8 * i + g, 0) + c * (D / 2);
#pragma unroll
            for (int j = 0; j < KH; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint4 w = *reinterpret_cast<const uint4*>(p + 32 * j + 16 * u);
                    kw[i][8 * j + 4 * u] = w.x; kw[i][8 * j + 4 * u + 1] = w.y;
                    kw[i][8 * j + 4 * u + 2] = w.z; kw[i][8 * j + 4 * u + 3] = w.w;
                }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bool bad;
            uint32_t mx = bf16_amax(kw[i], bad, true);
            mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
            mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
            const int e = bits_exp(mx);
            aa[0][i] = exp2i(e);
            ks[i] = exp2i(-e);
        }
#pragma unroll
        for (int u = 0; u < KH * 4; ++u) {
            uint32_t b[NQ][2];
            columns(qf, u, lane, b);
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                mma16816(s[0][q], bf16_f16(kw[0][2 * u], ks[0]), bf16_f16(kw[1][2 * u], ks[1]), bf16_f16(kw[0][2 * u + 1], ks[0]),
                         bf16_f16(kw[1][2 * u + 1], ks[1]), b[q][0], b[q][1]);
        }
        bool wide = false;
        int vx[4];                                        // exponents of keys 2c, 2c + 1, 2c + 8, 2c + 9
        uint32_t vw[4][VW * 2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = tok + 2 * c + (j & 1) + (j >> 1) * 8;
            const char* p = row(e, 1) + g * (D / 4);
#pragma unroll
            for (int u = 0; u < VW / 2; ++u) {
                const uint4 w = *reinterpret_cast<const uint4*>(p + 16 * u);
                vw[j][4 * u] = w.x; vw[j][4 * u + 1] = w.y; vw[j][4 * u + 2] = w.z; vw[j][4 * u + 3] = w.w;
            }
            bool bad;
            uint32_t mx = bf16_amax(vw[j], bad, false);
            if (bad && e < keys) atomicOr(&bad_v[e >> 5], 1u << (e & 31));
#pragma unroll
            for (int d = 4; d < 32; d *= 2) mx = max(mx, __shfl_xor_sync(FULL, mx, d));
            const int ex = bits_exp(mx);
            vx[j] = ex;
            wide |= e < keys && is_far_exp(ex);
#pragma unroll
            for (int u = 0; u < VW * 2; ++u) vw[j][u] = bf16_f16(vw[j][u], exp2i(-ex));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {                     // of keys g and g + 8
            const int even = __shfl_sync(FULL, vx[2 * i], g >> 1), odd = __shfl_sync(FULL, vx[2 * i + 1], g >> 1);
            const int ex = g & 1 ? odd : even;
            bb[0][i] = (float)ex;
            ii[0][i] = exp2i(-ex);
        }
        uint32_t mask[NQ][2], p[1][NQ][2];
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) mask[q][e] = tail_bits(P, sg.b, min(8 * q + 2 * c + e, P.R - 1) / P.G, sg.q.open, tok) & 0xffffu;
        if (far || __any_sync(FULL, wide)) {
            if (!far) go_far();
            far_sums<1, true>(s, rq, aa, mask);
            ii[0][0] = ii[0][1] = 0.f;
        }
        softmax<1, true>(s, rq, aa, bb, ii, mask, p);
#pragma unroll
        for (int u = 0; u < VW * 2; ++u) {
            uint32_t x[2], y[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x[h] = __byte_perm(vw[0][u], vw[1][u], h ? 0x7632 : 0x5410);
                y[h] = __byte_perm(vw[2][u], vw[3][u], h ? 0x7632 : 0x5410);
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) mma16816(o[q][u], x[0], x[1], y[0], y[1], p[0][q][0], p[0][q][1]);
        }
    }
    // The item's queries as fragments, and the factors of this lane's columns.
    __device__ __forceinline__ void load_q(const Seg& sg, uint32_t* qf, float (&rq)[NQ][2]) {
        uint32_t w[NQ][KH * 8];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int row = min(g + 8 * q, P.R - 1), n = row / P.G;
            const char* p = P.q.p + sg.b * P.q.b + n * P.q.n + (sg.h * P.G + row - n * P.G) * P.q.h + c * (D / 2);
#pragma unroll
            for (int j = 0; j < KH; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint4 v = *reinterpret_cast<const uint4*>(p + 32 * j + 16 * u);
                    w[q][8 * j + 4 * u] = v.x; w[q][8 * j + 4 * u + 1] = v.y;
                    w[q][8 * j + 4 * u + 2] = v.z; w[q][8 * j + 4 * u + 3] = v.w;
                }
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            bool bad;
            uint32_t mx = bf16_amax(w[q], bad, true);
            mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
            mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
            const int ex = bits_exp(mx);                  // of query 8q + g
            const float sc = exp2i(-ex);
#pragma unroll
            for (int e = 0; e < 2; ++e) rq[q][e] = exp2i(__shfl_sync(FULL, ex, 4 * (2 * c + e))) * P.scale;
#pragma unroll
            for (int u = 0; u < KH * 4; ++u) {
                qf[(u * 32 + lane) * 2 * NQ + 2 * q] = bf16_f16(w[q][2 * u], sc);
                qf[(u * 32 + lane) * 2 * NQ + 2 * q + 1] = bf16_f16(w[q][2 * u + 1], sc);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) o[q][j][0] = o[q][j][1] = o[q][j][2] = o[q][j][3] = 0.f;
            m[q][0] = m[q][1] = NEG_INF;
            l[q][0] = l[q][1] = 0.f;
        }
        far = false;
        __syncwarp();
    }
};

template <int D, int NQ> struct alignas(16) MmShared {
    MmRing<D> ring[MM_WARPS];                             // 1024-byte aligned, as the swizzle wants
    MmSlots slots[MM_WARPS];
    alignas(16) uint32_t q[D / 16 * 32 * 2 * NQ];         // the query fragments: every warp writes the same
    float4 o[2][4][32];                                   // output fragments of two warps, four blocks at a time
    float m[MM_WARPS][8 * NQ], l[MM_WARPS][8 * NQ];
    uint32_t bad_v[12];
    int bad;
    MmAhead now, ahead[MM_WARPS];                         // the segment being computed; of each warp's next chunk
};

// The end of a segment: the warps' results put together and written out, or left as a part.
template <int D, int NQ>
__device__ __forceinline__ void mm_finish(const Att& P, MmWarp<D, NQ>& w, MmShared<D, NQ>& sh, bool bad) {
    const int tid = threadIdx.x;
    const Seg& g = sh.now.s;
    constexpr int NT = D / 16;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d *= 2) w.l[q][e] += __shfl_xor_sync(FULL, w.l[q][e], d);
            if (w.g == 0) {
                sh.m[w.warp][8 * q + 2 * w.c + e] = w.m[q][e];
                sh.l[w.warp][8 * q + 2 * w.c + e] = w.l[q][e];
                if (!w.far) w.ref[8 * q + 2 * w.c + e] = w.own_ref(q, e);
            }
        }
    if (bad) sh.bad = 1;
    __syncthreads();
    // every warp's output on the common maximum, then warps 2 and 3 to 0 and 1, and 1 to 0
    float mm[NQ][2], l[NQ][2], rr[NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = 8 * q + 2 * w.c + e;
            mm[q][e] = fmaxf(fmaxf(sh.m[0][row], sh.m[1][row]), fmaxf(sh.m[2][row], sh.m[3][row]));
            const float base = mm[q][e] == NEG_INF ? 0.f : mm[q][e], f = ex2(w.m[q][e] - base);
            const float ri[MM_WARPS] = {sh.slots[0].ref[row], sh.slots[1].ref[row], sh.slots[2].ref[row], sh.slots[3].ref[row]};
            rr[q][e] = fmaxf(fmaxf(ri[0], ri[1]), fmaxf(ri[2], ri[3]));
            const float ref = rr[q][e] == NEG_INF ? 0.f : rr[q][e];
            l[q][e] = 0.f;
#pragma unroll
            for (int i = 0; i < MM_WARPS; ++i) l[q][e] = fmaf(ex2(ri[i] - ref), sh.l[i][row], l[q][e]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                w.o[q][j][e] *= f;
                w.o[q][j][2 + e] *= f;
            }
        }
#pragma unroll
    for (int half = 2; half >= 1; half /= 2)
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int j0 = 0; j0 < NT; j0 += 4) {
                if (w.warp >= half && w.warp < 2 * half) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sh.o[w.warp - half][j][w.lane] =
                            make_float4(w.o[q][j0 + j][0], w.o[q][j0 + j][1], w.o[q][j0 + j][2], w.o[q][j0 + j][3]);
                }
                __syncthreads();
                if (w.warp < half) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 x = sh.o[w.warp][j][w.lane];
                        w.o[q][j0 + j][0] += x.x; w.o[q][j0 + j][1] += x.y; w.o[q][j0 + j][2] += x.z; w.o[q][j0 + j][3] += x.w;
                    }
                }
                __syncthreads();
            }
    const bool whole = g.whole();
    const bool nan = g.q.bad || sh.bad;
    const float quiet = __int_as_float(0x7fffffff);
    if (w.warp == 0) {
        float* part = partial_of<D>(P, blockIdx.x, g.t0 == 0 ? 1 : 0);
        uint32_t any_bad = 0;
        if (g.t1 > g.q.nct)
            for (int i = 0; i < 12; ++i) any_bad |= sh.bad_v[i];
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = 8 * q + 2 * w.c + e, n = row / P.G;
            if (row >= P.R) continue;
            float x[2 * NT];                              // dims from g D / 8 on
#pragma unroll
            for (int j = 0; j < 2 * NT; ++j) x[j] = w.o[q][j >> 1][2 * (j & 1) + e];
            if (any_bad) {                                // values that could not enter the product
                for (int i = 0; i < 12; ++i) {
                    uint32_t hit = sh.bad_v[i];
                    if (hit) hit &= tail_bits(P, g.b, n, g.q.open, 32 * i);
                    for (; hit; hit &= hit - 1) {
                        const int k = 32 * i + __ffs(hit) - 1;
                        const char* src = k < g.q.open
                            ? static_cast<const char*>(P.c.v_open) +
                                  (((int64_t)g.q.slot * P.Hkv + g.h) * 2 * P.page + (g.q.full + k) % (2 * P.page)) * D * 2
                            : P.v.p + g.b * P.v.b + (k - g.q.open) * P.v.n + g.h * P.v.h;
                        const __nv_bfloat16* vv = reinterpret_cast<const __nv_bfloat16*>(src) + 2 * w.g * NT;
#pragma unroll
                        for (int j = 0; j < 2 * NT; ++j) {
                            const float y = __bfloat162float(vv[j]);
                            if (!(fabsf(y) <= 3.402823466e38f)) x[j] += y;
                        }
                    }
                }
            }
            const int64_t at = ((int64_t)g.b * P.N + n) * P.Hq + g.h * P.G + row - n * P.G;
            const float m = mm[q][e] == NEG_INF ? NEG_INF : mm[q][e] - P_BIAS, r = rr[q][e], sum = l[q][e];
            if (whole) {
                const float up = half_exp2(m == NEG_INF ? 0.f : m - r), inv = (nan ? quiet : sum == 0.f ? 0.f : 1.f / sum) * up;
#pragma unroll
                for (int j = 0; j < 2 * NT; ++j) x[j] = x[j] * up * inv;
                char* dst = P.out + (at * D + 2 * w.g * NT) * 2;
#pragma unroll
                for (int j = 0; j < 2 * NT; j += 8)
                    *reinterpret_cast<uint4*>(dst + 2 * j) =
                        make_uint4(pack_bf16(x[j], x[j + 1]), pack_bf16(x[j + 2], x[j + 3]),
                                   pack_bf16(x[j + 4], x[j + 5]), pack_bf16(x[j + 6], x[j + 7]));
                if (w.g == 0 && P.lse) P.lse[at] = nan ? quiet : sum == 0.f ? NEG_INF : (r + log2f(sum)) * LN2;
            } else {
                float* dst = part + (int64_t)row * D + 2 * w.g * NT;
#pragma unroll
                for (int j = 0; j < 2 * NT; j += 4)
                    *reinterpret_cast<float4*>(dst + j) =
                        nan ? make_float4(quiet, quiet, quiet, quiet) : make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                if (w.g == 0) {
                    float* stat = part + (int64_t)P.R * D + row;
                    stat[0] = m;
                    stat[P.R] = nan ? quiet : m == r ? sum : -sum;
                    if (m != r) stat[2 * P.R] = r;
                }
            }
        }
    }
    if (tid == 0) {
        if (nan) atomicOr(P.status, 1u << SPEC_ERR_DEVICE_INPUT);
        if (!whole && g.t0 == 0) P.cut[blockIdx.x] = Cut{g.b, g.h, g.mt, parts_of(P, g, sh.now.it.s, blockIdx.x)};
    }
    __syncthreads();
    if (tid < 12) sh.bad_v[tid] = 0;
    if (tid == 12) sh.bad = 0;
    if (tid == 32) sh.now.more = sh.now.it.next(P, sh.now.s);
    __syncthreads();
}

template <int D, int NQ>
__global__ void __launch_bounds__(MM_BT, MM_CTAS_SM) k_attention_mma(const Att P, const __grid_constant__ CUtensorMap kmap,
                                                                     const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ unsigned char mm_smem[];
    MmShared<D, NQ>& sh = *reinterpret_cast<MmShared<D, NQ>*>(mm_smem + (-smem_u32(mm_smem) & 1023u));
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Stretch st = find_stretch<MM_BT>(P);
    if (threadIdx.x == 0) P.cut[blockIdx.x].parts = 0;
    if (st.lo >= st.hi) return;
    if (threadIdx.x < 12) sh.bad_v[threadIdx.x] = 0;
    if (threadIdx.x == 12) sh.bad = 0;
    if (threadIdx.x == 32) {
        sh.now.it.begin(P, st);
        sh.now.more = sh.now.it.next(P, sh.now.s);
    }
    if (threadIdx.x == 64) {
        for (int i = 0; i < MM_WARPS * 2; ++i) bar_init(&sh.slots[i >> 1].full[i & 1], 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        proxy_fence();
    }
    __syncthreads();
    MmWarp<D, NQ> w(P, threadIdx.x >> 5, sh.ahead[threadIdx.x >> 5], sh.slots[threadIdx.x >> 5]);
    MmRing<D>& ring = sh.ring[w.warp];
    MmSlots& slots = sh.slots[w.warp];
    w.begin(st);
    uint32_t* qf = sh.q;
    float rq[NQ][2];
    int id, idy, parity = -1;
    // part x is computed, y's bytes are on their way, and the page ids of the part after
    Part x = w.next(id);
    w.fetch(x, id, 0, ring, slots, &kmap, &vmap);
    Part y{};
    idy = -2;
    if (x.kind()) y = w.next(idy);
    bool bad = false, lost = false;                       // lost: a copy that did not land; nothing is sent after it
    unsigned full = 0;                                    // parity of each slot's next phase
    for (int s = 0; x.kind(); s ^= 1) {
        if (!lost) w.fetch(y, idy, s ^ 1, ring, slots, &kmap, &vmap);
        if (x.parity() != parity) {
            parity = x.parity();
            w.load_q(sh.now.s, qf, rq);
        }
        Part z{};
        int idz = -2;
        if (y.kind()) z = w.next(idz);
        if (x.kind() == 1) {
            const bool came = !lost && P.wait_tries != 0 &&
                              (bar_try(&slots.full[s], full >> s & 1) || bar_wait_slow(&slots.full[s], full >> s & 1, nullptr, P.wait_tries));
            if (!__all_sync(FULL, came)) {
                bad = true;
                if (!lost) {                              // let them land (bounded), whatever becomes of the result
                    bool landed = bar_wait_slow(&slots.full[s], full >> s & 1, nullptr);
                    if (y.kind() == 1) landed &= bar_wait_slow(&slots.full[s ^ 1], full >> (s ^ 1) & 1, nullptr);
                    lost = __any_sync(FULL, !landed);
                    if (w.lane == 0) atomicOr(P.status, (1u << SPEC_ERR_TIMEOUT) | (lost ? 1u << SPEC_ERR_COPY_IN_FLIGHT : 0u));
                }
            }
            full ^= 1u << s;
            const unsigned there = __ballot_sync(FULL, id >= 0 && id < P.c.num_pages) & 3u, none = __ballot_sync(FULL, id == -2) & 3u;
            bad |= (there | none) != 3u;
            if (there == 3u) w.template cached<2>(ring, slots, s, qf, rq);
            else if (there == 1u) w.template cached<1>(ring, slots, s, qf, rq);
        } else if (x.kind() == 2) {
#pragma unroll 1
            for (int n = 0; n < 2; ++n) {
                const int tok = x.tok + w.first_key(n);
                if (tok < sh.now.s.q.open + P.N) w.tail(tok, sh.now.s, qf, rq, sh.bad_v);
            }
        }
        if (y.kind() == 0 || y.parity() != x.parity()) {
            mm_finish<D, NQ>(P, w, sh, bad);
            bad = false;
        }
        x = y;
        y = z;
        id = idy;
        idy = idz;
    }
}

}  // namespace

using sv_host::fail;

namespace {

// What an item costs on the line of work beside its tiles, in tiles (its start, its end, its cut).  64 chains of 6 over ragged
// lengths up to 4096 took 217, 209, 203 us at 2, 3, 4 (an earlier form 268 at 8), 32 trees of 64 over 8192 575, 553, 543 (635);
// 64 single tokens over 8192 118, 117, 122.
constexpr int TC_OVER = 4, MM_OVER = 3;
constexpr int TC_CTAS = 148, MM_CTAS = MM_CTAS_SM * 148;      // CTAs at most

template <int D>
spec_status launch_merge(const Att& P, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, (unsigned)((P.R < 256 ? P.R : 256) + MERGE_ROWS - 1) / MERGE_ROWS);
    cfg.blockDim = dim3(MERGE_BT);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_attention_merge<D>, P);
    if (e != cudaSuccess) return fail(SPEC_ERR_CUDA, "k_attention_merge launch: %s", cudaGetErrorString(e));
    return sv_host::launched("k_attention_merge");
}

// The cache's keys or values as a matrix of 8-bit rows; a box of `rows` of them (a page of one head, or a part of it).
template <int D>
spec_status page_map(const Att& P, void* pages, int rows, CUtensorMap* map) {
    static std::atomic<void*> entry{nullptr};
    void* f = entry.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess || found != cudaDriverEntryPointSuccess || !f)
            return fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
        entry.store(f, std::memory_order_release);
    }
    const bool empty = P.c.num_pages == 0;                // nothing is copied then: any address serves
    const cuuint64_t dims[2] = {(cuuint64_t)D, empty ? (cuuint64_t)P.page : (cuuint64_t)P.c.num_pages * P.Hkv * P.page};
    const cuuint64_t strides[1] = {(cuuint64_t)D};
    const cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)rows}, step[2] = {1, 1};
    const CUresult r = reinterpret_cast<CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)>(f)(
        map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, empty ? static_cast<void*>(P.out) : pages, dims, strides, box, step,
        CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", (int)r);
    return SPEC_OK;
}

template <int D>
spec_status launch_tc(Att P, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    P.over = TC_OVER;
    if (const spec_status s = sv_host::allow_smem(reinterpret_cast<const void*>(k_attention_tc<D>), "k_attention_tc", tc_smem<D>(), done)) return s;
    const int ctas = sv_host::num_sms() < TC_CTAS ? sv_host::num_sms() : TC_CTAS;
    CUtensorMap kmap;
    if (const spec_status s = page_map<D>(P, P.c.k_pages, P.page, &kmap)) return s;
    k_attention_tc<D><<<ctas, TC_BT, tc_smem<D>(), st>>>(P, kmap);
    const spec_status s = sv_host::launched("k_attention_tc");
    return s == SPEC_OK ? launch_merge<D>(P, ctas, st) : s;
}

template <int D, int NQ>
spec_status launch_mma(Att P, cudaStream_t st) {
    const size_t smem = sizeof(MmShared<D, NQ>) + 1024;
    static std::atomic<uint64_t> done{0};
    P.over = MM_OVER;
    if (const spec_status s = sv_host::allow_smem(reinterpret_cast<const void*>(k_attention_mma<D, NQ>), "k_attention_mma", smem, done)) return s;
    CUtensorMap kmap, vmap;
    if (const spec_status s = page_map<D>(P, P.c.k_pages, 16, &kmap)) return s;
    if (const spec_status s = page_map<D>(P, P.c.v_pages, 16, &vmap)) return s;
    const int want = MM_CTAS_SM * sv_host::num_sms(), ctas = want < MM_CTAS ? want : MM_CTAS;
    k_attention_mma<D, NQ><<<ctas, MM_BT, smem, st>>>(P, kmap, vmap);
    const spec_status s = sv_host::launched("k_attention_mma");
    return s == SPEC_OK ? launch_merge<D>(P, ctas, st) : s;
}

template <int D>
spec_status launch(const Att& P, cudaStream_t st) {
    if (P.R > MM_ROWS) return launch_tc<D>(P, st);
    return P.R > 8 ? launch_mma<D, 2>(P, st) : launch_mma<D, 1>(P, st);
}

}  // namespace

extern "C" {

size_t spec_cache_workspace_bytes(int B, int N, int q_heads, int head_dim) {
    if (B < 0 || B > sv_host::CACHE_MAX_B || N < 1 || N > SPEC_MAX_NODES || q_heads < 1 || q_heads > SPEC_MAX_HEADS ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    // rows of an item: at most N * q_heads (one kv head), 16 of them in the kernel with more CTAs
    const size_t rows = (size_t)N * q_heads < 256 ? (size_t)N * q_heads : 256, few = rows < MM_ROWS ? rows : MM_ROWS;
    const size_t tc = 2 * TC_CTAS * partial_floats(rows, head_dim), mm = 2 * MM_CTAS * partial_floats(few, head_dim);
    return sv_host::CACHE_WS_PARTIAL + sv_host::align256(sizeof(float) * (tc > mm ? tc : mm));
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
    P.B = B; P.N = N; P.Hq = q_heads; P.Hkv = cache->kv_heads; P.G = q_heads / cache->kv_heads;
    P.R = N * P.G;
    P.mtiles = (P.R + 255) / 256;
    P.page = cache->page_size;
    P.pshift = __builtin_ctz(P.page);
    P.c = *cache;
    P.anc = reinterpret_cast<const uint32_t*>(ancestors);
    P.scale = (float)((double)scale * 1.4426950408889634073599);
    P.out = static_cast<char*>(out);
    P.lse = lse;
    char* ws = static_cast<char*>(workspace);
    P.status = reinterpret_cast<unsigned*>(ws + sv_host::CACHE_WS_STATUS);
    P.wait_tries = sv_host::wait_tries();
    P.cut = reinterpret_cast<Cut*>(ws + sv_host::CACHE_WS_CUT);
    P.partial = reinterpret_cast<float*>(ws + sv_host::CACHE_WS_PARTIAL);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return D == 64 ? launch<64>(P, st) : launch<128>(P, st);
}

}  // extern "C"
