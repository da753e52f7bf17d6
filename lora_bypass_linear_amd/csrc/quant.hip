// quant.hip -- e4m3 codes with one fp32 scale per group: rows of activations
// in groups of 128, weights in 128 x 128 tiles.
//
//   s = max(amax, 2^-100) / 448        one correctly rounded fp32 division
//   q = e4m3(x / s)                    the exact quotient rounded once, ties to even
//
// The quotient's rounding has to be exact: with 16-bit inputs x / amax is a
// ratio of small integers, so x / s lies within a rounding of s of a midpoint
// between codes for a share of all elements that no tolerance hides, and an
// approximate quotient would give other codes from build to build.
//
// Bound by memory (es + 1 bytes an element); the exact quotient costs about a
// dozen vector operations an element, which the loads in flight cover.
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
template <int DT>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantRowsParams p, int pairs) {
    const int tid = threadIdx.x;
    const int64_t m = ((int64_t)blockIdx.x / pairs) * 16 + (tid >> 4);
    const int64_t kb = ((int64_t)blockIdx.x % pairs) * 2 + ((tid >> 3) & 1);
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

// One 128 x 128 tile per workgroup: 8 lanes a row, 4 passes of 32 rows kept
// in registers, one maximum over the workgroup, then the codes; the
// transposed codes go through LDS (rows of 132 bytes: consecutive rows start
// one bank apart).
template <int DT>
__global__ __launch_bounds__(256) void quant_tiles_kernel(QuantTilesParams p, int kblocks) {
    constexpr int LD = 132;
    __shared__ uint32_t wmax[4];
    __shared__ __attribute__((aligned(16))) uint8_t t[128 * LD];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t nb = (int64_t)blockIdx.x / kblocks, kb = (int64_t)blockIdx.x % kblocks;
    const int64_t n0 = nb * FP8_BLOCK, k0 = kb * FP8_BLOCK;
    const int c = (tid & 7) * 16;
    Raw16<DT> x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = n0 + i * 32 + (tid >> 3);
        if (n < p.N && k0 + c < p.K) x[i].load(p.w, n * p.K + k0 + c);
        else x[i].zero();
    }
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) b = umax(b, x[i].amax_bits());
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) b = umax(b, (uint32_t)__shfl_xor((int)b, d));
    if (lane == 0) wmax[wave] = b;
    __syncthreads();
    b = umax(umax(wmax[0], wmax[1]), umax(wmax[2], wmax[3]));
    const float s = scale_of(b), inv = __builtin_amdgcn_rcpf(s);
    if (tid == 0) p.s[nb * kblocks + kb] = s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 32 + (tid >> 3);
        const i32x4 q = x[i].codes(s, inv);
        if (p.q != nullptr && n0 + r < p.N && k0 + c < p.K) *(i32x4*)((char*)p.q + (n0 + r) * p.K + k0 + c) = q;
        if (p.q_t != nullptr) {
            uint32_t* d = (uint32_t*)(t + r * LD + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = (uint32_t)q[e];
        }
    }
    if (p.q_t == nullptr) return;
    __syncthreads();
    // 16 rows of one column are 16 consecutive bytes of a row of q_t
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = i * 32 + (tid >> 3), r0 = (tid & 7) * 16;
        i32x4 o;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) w |= (uint32_t)t[(r0 + 4 * g + e) * LD + k] << (8 * e);
            o[g] = (int)w;
        }
        if (k0 + k < p.K && n0 + r0 < p.N) *(i32x4*)((char*)p.q_t + (k0 + k) * p.N + n0 + r0) = o;
    }
}

hipError_t launch_quant_rows(const QuantRowsParams& p, hipStream_t s) {
    if (p.M <= 0 || p.K <= 0) return hipSuccess;
    const int pairs = (int)((p.K + 2 * FP8_BLOCK - 1) / (2 * FP8_BLOCK));
    const int64_t wgs = (p.M + 15) / 16 * pairs;
    if (wgs >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    const dim3 g((unsigned)wgs);
    if (p.x_dt == DT_F32) hipLaunchKernelGGL(quant_rows_kernel<DT_F32>, g, dim3(256), 0, s, p, pairs);
    else if (p.x_dt == DT_F16) hipLaunchKernelGGL(quant_rows_kernel<DT_F16>, g, dim3(256), 0, s, p, pairs);
    else hipLaunchKernelGGL(quant_rows_kernel<DT_BF16>, g, dim3(256), 0, s, p, pairs);
    return hipGetLastError();
}

hipError_t launch_quant_tiles(const QuantTilesParams& p, hipStream_t s) {
    if (p.N <= 0 || p.K <= 0) return hipSuccess;
    const int kblocks = (int)((p.K + FP8_BLOCK - 1) / FP8_BLOCK);
    const int64_t wgs = (p.N + FP8_BLOCK - 1) / FP8_BLOCK * kblocks;
    if (wgs >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    const dim3 g((unsigned)wgs);
    if (p.w_dt == DT_F32) hipLaunchKernelGGL(quant_tiles_kernel<DT_F32>, g, dim3(256), 0, s, p, kblocks);
    else if (p.w_dt == DT_F16) hipLaunchKernelGGL(quant_tiles_kernel<DT_F16>, g, dim3(256), 0, s, p, kblocks);
    else hipLaunchKernelGGL(quant_tiles_kernel<DT_BF16>, g, dim3(256), 0, s, p, kblocks);
    return hipGetLastError();
}

}  // namespace lyc
