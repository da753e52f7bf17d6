// bwd.hip -- the transposed copies the LoRA-bypass backward contracts over
// tokens with.  dDown = gh_r^T . x_c and dUp = scale * dy_c^T . h_r sum over
// the token index, which is the row index of x, dy, h_r and gh_r; the GEMM
// reads both operands along their rows, so those four (and W for
// dx = dy_c . W_c) are first copied transposed, rounded to the compute dtype,
// with zero padding to 8-element rows.
#include "bwd.h"
#include "lyc_device.h"
#include "quant_device.h"
#include "transpose_device.h"

namespace lyc {

template <class T>
__global__ __launch_bounds__(256) void transpose_kernel(TransposeParams p, int64_t tiles_r) {
    __shared__ float t[64][65];
    transpose_body<T>(p, blockIdx.x, tiles_r, t);
}

// What the backward over an 8-bit base prepares, in one launch: up^T, down^T
// (workgroups below na, below nb) and dy quantized (the rest): 5 us at 300 x
// 1040 x 2064, rank 5, against 11 in three launches.
template <class T, int DT>
__global__ __launch_bounds__(256) void bwd_prep_kernel(TransposeParams u, TransposeParams d, QuantRowsParams q, unsigned na,
                                                       unsigned nb, int pairs) {
    __shared__ float t[64][65];
    if (blockIdx.x < na) transpose_body<T>(u, blockIdx.x, (u.rows_pad + 63) / 64, t);
    else if (blockIdx.x < nb) transpose_body<T>(d, blockIdx.x - na, (d.rows_pad + 63) / 64, t);
    else quant_rows_body<DT>(q, blockIdx.x - nb, pairs);
}

template <class T>
static hipError_t run_bwd_prep(const TransposeParams& u, const TransposeParams& d, const QuantRowsParams& q,
                               hipStream_t s) {
    const int pairs = quant_pairs(q.K);
    const int64_t na = transpose_tiles(u), nb = na + transpose_tiles(d), all = nb + (q.M + 15) / 16 * pairs;
    if (all >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    const dim3 g((unsigned)all);
    if (q.x_dt == DT_F32)
        hipLaunchKernelGGL((bwd_prep_kernel<T, DT_F32>), g, dim3(256), 0, s, u, d, q, (unsigned)na, (unsigned)nb, pairs);
    else if (q.x_dt == DT_F16)
        hipLaunchKernelGGL((bwd_prep_kernel<T, DT_F16>), g, dim3(256), 0, s, u, d, q, (unsigned)na, (unsigned)nb, pairs);
    else
        hipLaunchKernelGGL((bwd_prep_kernel<T, DT_BF16>), g, dim3(256), 0, s, u, d, q, (unsigned)na, (unsigned)nb, pairs);
    return hipGetLastError();
}

hipError_t launch_bwd_prep(const TransposeParams& u, const TransposeParams& d, const QuantRowsParams& q, hipStream_t s) {
    if ((u.src_dt == DT_F32) != (d.src_dt == DT_F32)) return hipErrorInvalidValue;
    return u.src_dt == DT_F32 ? run_bwd_prep<uint32_t>(u, d, q, s) : run_bwd_prep<uint16_t>(u, d, q, s);
}

hipError_t launch_transpose(const TransposeParams& p, hipStream_t s) {
    if (p.rows_pad <= 0 || p.cols_pad <= 0) return hipSuccess;
    const int64_t tr = (p.rows_pad + 63) / 64, tc = (p.cols_pad + 63) / 64;
    const dim3 grid((unsigned)(tr * tc));
    if (p.src_dt == DT_F32) hipLaunchKernelGGL(transpose_kernel<uint32_t>, grid, dim3(256), 0, s, p, tr);
    else hipLaunchKernelGGL(transpose_kernel<uint16_t>, grid, dim3(256), 0, s, p, tr);
    return hipGetLastError();
}

}  // namespace lyc
