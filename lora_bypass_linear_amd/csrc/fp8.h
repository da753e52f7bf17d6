// fp8.h -- host-side launchers of the 8-bit (OCP e4m3) base-weight kernels
// (internal to the library; the public surface is include/lyc.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace lyc {

constexpr int FP8_BLOCK = 128;   // elements a scale covers along each blocked axis

// q[m][k] = e4m3(x[m][k] / s), s[k / 128][m] = max(|x| over the group, 2^-100) / 448
struct QuantRowsParams {
    const void* x;   // [M][K] in x_dt, 16-byte aligned; K a multiple of 16
    int x_dt;
    void* q;         // [M][K] e4m3 codes, 16-byte aligned
    float* s;        // [ceil(K/128)][M]
    int64_t M, K;
};
hipError_t launch_quant_rows(const QuantRowsParams& p, hipStream_t s);
inline int quant_pairs(int64_t K) { return (int)((K + 2 * FP8_BLOCK - 1) / (2 * FP8_BLOCK)); }
// the few-row h pass and the quantization of the same x in one launch (x in
// the 16-bit compute dtype), hpass.hip
hipError_t launch_hdot_quant(int c_dt, const HdotParams& h, const QuantRowsParams& q, hipStream_t s);

// the same with one scale per 128 x 128 tile, s[n / 128][k / 128]; q and the
// transposed codes q_t [K][N] (N a multiple of 16) may each be nullptr
struct QuantTilesParams {
    const void* w;   // [N][K] in w_dt, 16-byte aligned; K a multiple of 16
    int w_dt;
    void* q;
    void* q_t;
    float* s;
    int64_t N, K;
};
hipError_t launch_quant_tiles(const QuantTilesParams& p, hipStream_t s);

// y = round_out( scale * (af . bf^T) + sum_kb sx[kb][m] sw(n/128, kb) (a . b^T over block kb) + bias ):
// g.a = weight codes [N][K], g.b = activation codes [M][K] (K bytes a row, a
// multiple of 16), g.af / g.bf / g.rf the fold's operands in the compute dtype
// c_dt as in launch_gemm, sw(i, j) = sw[i * sw_n + j * sw_k].  g.gain, ta, tb,
// post and tile are not used.
struct Fp8GemmParams {
    GemmParams g;
    const float* sx;   // [ceil(K/128)][M]
    const float* sw;
    int64_t sw_n, sw_k;
};
hipError_t launch_fp8_gemm(int c_dt, const Fp8GemmParams& p, hipStream_t s);
// Output tile and K split launch_fp8_gemm takes (the partial sums of a split
// need ksplit * M * N * 4 bytes); up to 32 rows: the features and rows of a
// workgroup of the few-row kernel
struct Fp8Plan {
    int tile_n, tile_m, ksplit;
};
Fp8Plan fp8_gemm_plan(int64_t M, int64_t N, int64_t K, int y_dt);

// y = round_out(post * (the K splits' partial sums in split order) + bias), gemm.hip
hipError_t launch_gemm_reduce(const GemmParams& p, hipStream_t s);

}  // namespace lyc
