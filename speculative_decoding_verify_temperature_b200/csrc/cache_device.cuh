// cache_device.cuh -- device helpers of the cache kernels: rows in vectors of
// elements, the RMS norm and the rotation of a head row, e4m3.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_verify.h"

namespace svc {

constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {   // round to nearest, ties to even
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 bytes (lo in bits 0-7), round to nearest even, NaN -> 0x7F.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight consecutive bf16 elements as they lie in memory.
struct Bf16x8 {
    uint4 a;
    __device__ __forceinline__ void load(const char* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
};

// cos and sin of pos * f.  The angle is formed in f64, in turns, and reduced to
// [-1/2, 1/2] there: f32 would lose a far position's angle (at 2^20 its spacing
// is 2^-4 rad).
__device__ __forceinline__ float2 cos_sin(int pos, float f) {
    double t = (double)pos * ((double)f * 0.15915494309189533577);
    t -= rint(t);
    float s, c;
    sincospif((float)(2.0 * t), &s, &c);
    return make_float2(c, s);
}

// Four consecutive elements.
template <int DT> struct Quad;
template <> struct Quad<SPEC_BF16> {
    static constexpr int ESZ = 2;
    uint2 a;
    __device__ __forceinline__ void load(const char* p) { a = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void load_bf16(const char* p) { load(p); }
    __device__ __forceinline__ void zero() { a = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float* x) const { x[0] = bf_lo(a.x); x[1] = bf_hi(a.x); x[2] = bf_lo(a.y); x[3] = bf_hi(a.y); }
    __device__ __forceinline__ void set(const float* x) { a = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])); }
    __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<uint2*>(p) = a; }
};
template <> struct Quad<SPEC_F32> {
    static constexpr int ESZ = 4;
    float4 a;
    __device__ __forceinline__ void load(const char* p) { a = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void load_bf16(const char* p) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        a = make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
    }
    __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float* x) const { x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; }
    __device__ __forceinline__ void set(const float* x) { a = make_float4(x[0], x[1], x[2], x[3]); }
    __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<float4*>(p) = a; }
};

// A head row of D elements lies in D / 8 consecutive lanes of an aligned group
// of GW lanes, two quads (four consecutive elements) in each; the lanes behind
// hold zeros.  The quads are chosen so that both elements of a rotated pair are
// in one lane: quads l and l + rot / 8 where the pairs are half a rotation apart,
// neighbours elsewhere.  In both orders lane l turns the pairs 4l to 4l + 3.
struct Quads {
    int q0, q1;
    bool turns;
    __device__ __forceinline__ Quads(int l, int rot, bool interleaved) {
        const int n = rot / 8;
        turns = l < n;
        const bool split = turns && !interleaved;
        q0 = split ? l : 2 * l;
        q1 = split ? l + n : 2 * l + 1;
    }
};

// 1 / rms of the row, in every lane of the group; all lanes of the warp call it.
__device__ __forceinline__ float row_rms(const float (&x)[8], int GW, float inv_d, float eps) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    for (int o = GW >> 1; o; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
    return rsqrtf(fmaf(ss, inv_d, eps));
}

// Turn the lane's four pairs: (x[i], x[4 + i]), or neighbours.
__device__ __forceinline__ void row_rotate(float (&x)[8], const float4& c, const float4& s, bool interleaved) {
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * cc[i] - b * ss[i];
            x[2 * i + 1] = b * cc[i] + a * ss[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[i], b = x[4 + i];
            x[i] = a * cc[i] - b * ss[i];
            x[4 + i] = b * cc[i] + a * ss[i];
        }
    }
}

}  // namespace svc
