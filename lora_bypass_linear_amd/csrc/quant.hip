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
#include "quant_device.h"

namespace lyc {

template <int DT>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantRowsParams p, int pairs) {
    quant_rows_body<DT>(p, blockIdx.x, pairs);
}

// One 128 x 128 tile per workgroup: 8 lanes a row, 4 passes of 32 rows kept
// in registers, one maximum over the workgroup, then the codes; the
// transposed codes go through LDS (rows of 132 bytes: consecutive rows start
// one bank apart).  fp32 4096 x 4096 with the transposed codes: 18.2 us, 5.5 TB/s.
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
    const int pairs = quant_pairs(p.K);
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
