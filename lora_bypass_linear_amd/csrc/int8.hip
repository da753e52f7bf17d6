// int8.hip -- rows quantized to 8-bit integers, and the instances of the int8
// product and gated block (pair_tile.h).
//
//   s = max(amax, 2^-100) / 127      one correctly rounded fp32 division
//   q = rint(x / s)                  of the exact quotient, ties to even
//
// The quotient is never formed to more bits than fp32 gives: f = floor(x (1/s))
// is the quotient's floor or one beside it, and the sign of x - (f + 1/2) s, one
// fused multiply-add ((f + 1/2) s has no rounding of its own there), says on
// which side of the border between two codes x lies; 0 is the tie.
//
// Bound by memory: a workgroup a row (rows of up to 1024: a few lanes), up to
// 8192 elements of it in registers between its maximum and its codes, so that x
// is read once (the rest of a longer row a second time, from L2).  bf16 16384 x
// 8192: 70 us, 5.7 TB/s; 16384 x 16384: 152 us, 5.3 TB/s; 8192 x 14336: 70 us,
// 5.0 TB/s; fp32 4096 x 4096: 13.6 us.
#include "pair_tile.h"
#include "quant_device.h"

namespace lyc {

hipError_t launch_int8(int mode, const PairParams& p, hipStream_t s) {
    return mode == PAIR_ONE ? run_pair_ct<CI8, PAIR_ONE>(p, s) : run_pair_ct<CI8, PAIR_PAIR>(p, s);
}

constexpr float Q8_TOP = 127.f;

__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
    const uint32_t b = amax_bits > Q_FLOOR ? amax_bits : Q_FLOOR;
    return __fdiv_rn(__builtin_bit_cast(float, b), Q8_TOP);
}

// (a row that holds an infinity or a NaN has an infinite or NaN scale: codes 0)
__device__ __forceinline__ int int8_code(float x, float s, float inv) {
    const float f = __builtin_floorf(x * inv);
    const float d = __builtin_fmaf(-(f + 0.5f), s, x);
    const int lo = (int)f;
    return lo + (d > 0.f || (d == 0.f && (lo & 1)) ? 1 : 0);
}

template <int DT>
__device__ __forceinline__ i32x4 int8_codes(const Raw16<DT>& x, float s, float inv) {
    i32x4 o;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= ((uint32_t)int8_code(x.get(4 * g + e), s, inv) & 0xFFu) << (8 * e);
        o[g] = (int)w;
    }
    return o;
}

// One workgroup a row, CH chunks of 16 elements a thread kept in registers
// between the maximum and the codes; rows longer than 256 * 16 * CH are read
// twice (the second time mostly from L2).
template <int DT, int CH>
__global__ __launch_bounds__(256) void quant_int8_kernel(QuantInt8Params p) {
    __shared__ uint32_t wmax[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t m = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, row = m * p.K;
    if (m >= p.M) return;
    const int chunks = (int)(p.K / 16);
    Raw16<DT> x[CH];
    uint32_t b = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * 256 + tid;
        if (i < chunks) x[c].load(p.x, row + (int64_t)i * 16);
        else x[c].zero();
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) b = umax(b, x[c].amax_bits());
    for (int i = CH * 256 + tid; i < chunks; i += 256) {
        Raw16<DT> t;
        t.load(p.x, row + (int64_t)i * 16);
        b = umax(b, t.amax_bits());
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) b = umax(b, (uint32_t)__shfl_xor((int)b, d));
    if (lane == 0) wmax[wave] = b;
    __syncthreads();
    b = umax(umax(wmax[0], wmax[1]), umax(wmax[2], wmax[3]));
    const float s = int8_scale(b);
    const float inv = b >= 0x7F800000u ? 0.f : __builtin_amdgcn_rcpf(s);
    if (tid == 0) p.s[m] = s;
    i32x4* q = (i32x4*)((char*)p.q + row);
    if (b >= 0x7F800000u) {
        for (int i = tid; i < chunks; i += 256) q[i] = i32x4{0, 0, 0, 0};
        return;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * 256 + tid;
        if (i < chunks) q[i] = int8_codes<DT>(x[c], s, inv);
    }
    for (int i = CH * 256 + tid; i < chunks; i += 256) {
        Raw16<DT> t;
        t.load(p.x, row + (int64_t)i * 16);
        q[i] = int8_codes<DT>(t, s, inv);
    }
}

// Rows of up to 1024 elements: 2^lsh lanes a row, the fewest that hold it 16
// elements each, so 256 >> lsh rows a workgroup and no LDS.
template <int DT>
__global__ __launch_bounds__(256) void quant_int8_short_kernel(QuantInt8Params p, int lsh) {
    const int l = threadIdx.x & ((1 << lsh) - 1);
    const int64_t m = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) << (8 - lsh)) + (threadIdx.x >> lsh), row = m * p.K;
    const bool on = m < p.M && l < (int)(p.K / 16);
    Raw16<DT> x;
    if (on) x.load(p.x, row + l * 16);
    else x.zero();
    uint32_t b = x.amax_bits();
    for (int d = 1; d < 1 << lsh; d <<= 1) b = umax(b, (uint32_t)__shfl_xor((int)b, d));
    const bool finite = b < 0x7F800000u;
    const float s = int8_scale(b);
    if (m < p.M && l == 0) p.s[m] = s;
    if (!on) return;
    i32x4 q = i32x4{0, 0, 0, 0};
    if (finite) q = int8_codes<DT>(x, s, __builtin_amdgcn_rcpf(s));
    *(i32x4*)((char*)p.q + row + l * 16) = q;
}

// n workgroups over two grid dimensions: 2^32 threads in one of them do not launch
static dim3 rows_grid(int64_t n) {
    const int64_t gx = n < (1 << 22) ? n : 1 << 22;
    return dim3((unsigned)gx, (unsigned)((n + gx - 1) / gx));
}

template <int DT>
static hipError_t run_quant_int8(const QuantInt8Params& p, hipStream_t s) {
    // a workgroup a row, however short, is late with its loads: bf16 2^20 x 128 939 us,
    // 69-72 so; 2^17 x 1024 130, 69
    if (p.K <= 1024) {
        int lsh = 0;
        while (p.K > 16 << lsh) ++lsh;
        const int64_t per = 256 >> lsh;
        hipLaunchKernelGGL((quant_int8_short_kernel<DT>), rows_grid((p.M + per - 1) / per), dim3(256), 0, s, p, lsh);
        return hipGetLastError();
    }
    const dim3 g = rows_grid(p.M);
    if (p.K <= 4096) hipLaunchKernelGGL((quant_int8_kernel<DT, 1>), g, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((quant_int8_kernel<DT, 2>), g, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_quant_int8(const QuantInt8Params& p, hipStream_t s) {
    if (p.M <= 0) return hipSuccess;
    if (p.M >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    if (p.x_dt == DT_F32) return run_quant_int8<DT_F32>(p, s);
    if (p.x_dt == DT_F16) return run_quant_int8<DT_F16>(p, s);
    return run_quant_int8<DT_BF16>(p, s);
}

}  // namespace lyc
