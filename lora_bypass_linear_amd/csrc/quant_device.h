// quant_device.h -- device code of the e4m3 quantization (quant.hip holds what
// it computes and why).
#pragma once

#include "fp8.h"
#include "lyc_device.h"

namespace lyc {

constexpr float Q_TOP = 448.f;          // the largest e4m3 value
constexpr uint32_t Q_FLOOR = 0x0D800000u;   // 2^-100 as fp32 bits

// The scale of a group from the bits of its largest magnitude (bit order: a
// NaN above infinity above every number, so both reach the scale).
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const uint32_t b = amax_bits > Q_FLOOR ? amax_bits : Q_FLOOR;
    return __fdiv_rn(__builtin_bit_cast(float, b), Q_TOP);
}

// x / s rounded to odd in fp32 (truncated, the last bit set when inexact),
// which rounds to e4m3 as the exact quotient does.  y is within one ulp of the
// quotient after one correction; r = x - y s is then exact, its sign says
// whether y is past the quotient and r != 0 whether it is inexact.  A group
// that holds an infinity or a NaN (s infinite or NaN) gives NaN throughout.
__device__ __forceinline__ float quotient_odd(float x, float s, float inv) {
    const float a = __builtin_fabsf(x);
    float y = a * inv;
    y = __builtin_fmaf(__builtin_fmaf(-y, s, a), inv, y);
    const float r = __builtin_fmaf(-y, s, a);
    const int rb = __builtin_bit_cast(int, r);
    uint32_t u = __builtin_bit_cast(uint32_t, y) + (uint32_t)(rb >> 31);
    u |= (uint32_t)rb != 0u ? 1u : 0u;
    return __builtin_copysignf(__builtin_bit_cast(float, u), x);
}

__device__ __forceinline__ uint32_t codes4(const float (&v)[4]) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
    return (uint32_t)w;
}

// 16 consecutive elements of a row as fp32 bits
template <int DT>
struct Raw16 {
    static constexpr int V = DT == DT_F32 ? 4 : 2;   // 16-byte loads
    i32x4 v[V];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        const i32x4* src = (const i32x4*)((const char*)p + at * (DT == DT_F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = src[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i32x4{0, 0, 0, 0};
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (DT == DT_F32) {
            return __builtin_bit_cast(float, (uint32_t)v[e >> 2][e & 3]);
        } else {
            const uint32_t w = (uint32_t)v[e >> 3][(e >> 1) & 3];
            if constexpr (DT == DT_BF16) return __builtin_bit_cast(float, (e & 1) ? (w & 0xFFFF0000u) : (w << 16));
            else return f16_to_f32((uint16_t)((e & 1) ? (w >> 16) : w));
        }
    }
    __device__ __forceinline__ uint32_t amax_bits() const {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint32_t b = __builtin_bit_cast(uint32_t, get(e)) & 0x7FFFFFFFu;
            m = b > m ? b : m;
        }
        return m;
    }
    __device__ __forceinline__ i32x4 codes(float s, float inv) const {
        i32x4 o;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = quotient_odd(get(4 * g + e), s, inv);
            o[g] = (int)codes4(f);
        }
        return o;
    }
};

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// One group of 128 per 8 lanes, 16 elements a lane; a workgroup takes 16 rows
// x 2 groups, so that its scale writes are runs of 16 consecutive floats.
// bf16 16384 x 8192: 70 us, 5.8 TB/s of reads and writes (a plain copy: 5.2).
// (workgroup `wg` of 256 threads; pairs: pairs of groups a row)
template <int DT>
__device__ __forceinline__ void quant_rows_body(const QuantRowsParams& p, int64_t wg, int pairs) {
    const int tid = threadIdx.x;
    const int64_t m = (wg / pairs) * 16 + (tid >> 4);
    const int64_t kb = (wg % pairs) * 2 + ((tid >> 3) & 1);
    const int64_t k = kb * FP8_BLOCK + (tid & 7) * 16;
    const bool in = m < p.M && k < p.K;
    Raw16<DT> x;
    if (in) x.load(p.x, m * p.K + k);
    else x.zero();
    uint32_t b = x.amax_bits();
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) b = umax(b, (uint32_t)__shfl_xor((int)b, d));
    const float s = scale_of(b);
    if (in) {
        *(i32x4*)((char*)p.q + m * p.K + k) = x.codes(s, __builtin_amdgcn_rcpf(s));
        if ((tid & 7) == 0) p.s[kb * p.M + m] = s;
    }
}

}  // namespace lyc
