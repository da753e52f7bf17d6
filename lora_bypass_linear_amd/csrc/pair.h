// pair.h -- host-side launchers of the gated feed-forward block and of the
// 8-bit integer products (internal to the library; the public surface is
// include/lyc.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bwd.h"

namespace lyc {

// both projections' launches at once (hpass.hip, prep.hip)
struct HdotParams;
struct XrParams;
struct PrepParams;
hipError_t launch_hdot2(int c_dt, const HdotParams& a, const HdotParams& b, int64_t ld, hipStream_t s);
hipError_t launch_xr2(int c_dt, const XrParams& a, const XrParams& b, hipStream_t s);
hipError_t launch_prep2(const PrepParams& a, const PrepParams& b, hipStream_t s);

// activations of the gated block: x sigmoid(x); x Phi(x); its tanh form
enum { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_COUNT = 3 };

// internal dtype code of int8 operands (the public codes are 1 to 3)
constexpr int DT_I8 = 4;

// What the products of pair_tile.h compute, with A_h . B^T the fp32 (int8:
// exact 32-bit) sums over K and "proj_h" = scale * (bf_h . af_h^T) + b . a_h^T
// + bias_h (int8: the sum times sw_h[n] sx[m], no fold):
//   ONE    y = round_out(proj_0)
//   PAIR   y = round_out(act(proj_0) * proj_1), keep[h] = round_c(proj_h) where given
//   SEQ    y = round_out(sum_h (bf_h . af_h^T) + b_h . a_h^T)
enum { PAIR_ONE, PAIR_PAIR, PAIR_SEQ };
struct PairParams {
    const void* a[2];    // [N][K]; rows 16-byte aligned
    const void* b[2];    // [M][K] (b[1]: SEQ)
    const void* af[2];   // fold: [N][rf]
    const void* bf[2];   // [M][ldf], rf columns read
    int64_t ldf;
    int64_t M, N, K, rf;
    float scale;
    const void* bias[2];   // nullptr: none (both or neither)
    int bias_dt;
    const float* sx;       // int8: [M]
    const float* sw[2];    // int8: [N]
    int act;
    void* y;
    int y_dt;
    void* keep[2];         // [M][N] in the compute dtype, or nullptr (both)
    int ksplit;            // > 1: sums [ksplit][1 or 2][M][N] (32 bits each) in partial, joined by a second kernel
    void* partial;
};

// tile and K split by modelled time; up to 32 rows the features and rows of a
// workgroup of the few-row kernel (ksplit 1)
struct PairPlan {
    int tile_n, tile_m, ksplit;   // features x rows
};
PairPlan pair_plan(int mode, int c_dt, int64_t M, int64_t N, int64_t K);
// a launch holds fewer than 2^32 threads a grid dimension
bool pair_fits(int mode, int c_dt, int64_t M, int64_t N, int64_t K);

// c_dt: DT_F16, DT_BF16, DT_F32 (PAIR, SEQ) or DT_I8 (ONE, PAIR)
hipError_t launch_pair(int mode, int c_dt, const PairParams& p, hipStream_t s);

// q[m][k] = rint(x[m][k] / s[m]), s[m] = max(|x[m]|, 2^-100) / 127
struct QuantInt8Params {
    const void* x;   // [M][K] in x_dt, 16-byte aligned; K a multiple of 16
    int x_dt;
    void* q;         // [M][K], 16-byte aligned
    float* s;        // [M]
    int64_t M, K;
};
hipError_t launch_quant_int8(const QuantInt8Params& p, hipStream_t s);

// dg = round_c(dy * value * act'(gate)), dv = round_c(dy * act(gate)), all [M][N]
// (N a multiple of 8), and the second half of a saved h [M][2 r_pad] as rows of
// its own (h == nullptr: none)
struct GateGradParams {
    const void* dy;
    int dy_dt;
    const void *gate, *value;   // compute dtype, 16-byte aligned
    void *dg, *dv;
    int64_t n;                  // M * N
    int act;
    const void* h;
    void* hv;                   // [M][r_pad]
    int64_t M;
    int r_pad;
    uint8_t* open;              // 16-bit compute: [n / 8] marks of the elements left to 64 bits
    // up to four transposed copies made by workgroups of the same launch (sources
    // all of 16 or all of 32 bits)
    TransposeParams tr[4];
    int ntr;
};
hipError_t launch_gate_grad(int c_dt, const GateGradParams& p, hipStream_t s);

}  // namespace lyc
