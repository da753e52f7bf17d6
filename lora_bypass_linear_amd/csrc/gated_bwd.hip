// gated_bwd.hip -- the gated block's backward: the gradients of the two
// projections from the kept ones, and dx over both weights in one product
// (pair_tile.h, SEQ).
//
//   dg = round_c( dy * v * act'(g) )    dv = round_c( dy * act(g) )
//   dx = round_x( gh_g.down_g + gh_v.down_v + dg.W_g + dv.W_v )
#include "act.h"
#include "pair_tile.h"

namespace lyc {

hipError_t launch_seq(int c_dt, const PairParams& p, hipStream_t s) {
    if (c_dt == DT_F16) return run_pair_ct<CF16, PAIR_SEQ>(p, s);
    if (c_dt == DT_BF16) return run_pair_ct<CBF16, PAIR_SEQ>(p, s);
    return run_pair_ct<CF32, PAIR_SEQ>(p, s);
}

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
    if constexpr (DT == DT_F32) {
        const f32x4 a = ((const f32x4*)p)[2 * i], b = ((const f32x4*)p)[2 * i + 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
    } else {
        const i32x4 w = ((const i32x4*)p)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t u = (uint32_t)w[e];
            v[2 * e] = DT == DT_F16 ? f16_to_f32((uint16_t)u) : bf16_to_f32((uint16_t)u);
            v[2 * e + 1] = DT == DT_F16 ? f16_to_f32((uint16_t)(u >> 16)) : bf16_to_f32((uint16_t)(u >> 16));
        }
    }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
    if constexpr (DT == DT_F32) {
        ((f32x4*)p)[2 * i] = f32x4{v[0], v[1], v[2], v[3]};
        ((f32x4*)p)[2 * i + 1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        i32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = (int)(DT == DT_F16 ? pack_f16x2(v[2 * e], v[2 * e + 1]) : pack_bf16x2(v[2 * e], v[2 * e + 1]));
        ((i32x4*)p)[i] = w;
    }
}

// 8 elements per thread, the rows' shapes do not matter; bound by memory (five
// passes over M x N).  The last workgroups copy the second half of a saved h to
// rows of its own, which the product over the tokens reads.
template <int C, int G>
__global__ __launch_bounds__(256) void gate_grad_kernel(GateGradParams p, unsigned nb) {
    if (blockIdx.x >= nb) {
        const int64_t per = p.r_pad * (C == DT_F32 ? 4 : 2) / 16;   // 16-byte chunks of a half row
        const int64_t i = (int64_t)(blockIdx.x - nb) * 256 + threadIdx.x;
        if (i >= p.M * per) return;
        const int64_t m = i / per, c = i - m * per;
        ((i32x4*)p.hv)[i] = ((const i32x4*)p.h)[m * 2 * per + per + c];
        return;
    }
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.n / 8) return;
    float dy[8], g[8], v[8], dg[8], dv[8];
    load8<G>(p.dy, i, dy);
    load8<C>(p.gate, i, g);
    load8<C>(p.value, i, v);
    auto grads = [&](auto act) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float slope;
            const float a = act(g[e], &slope);
            dg[e] = dy[e] * v[e] * slope;
            dv[e] = dy[e] * a;
        }
    };
    if (p.act == ACT_GELU) {
        grads([](float x, float* s) { return act_gelu<true>(x, s); });
    } else {
        float a, b;
        act_coeffs(p.act, a, b);
        grads([=](float x, float* s) { return act_logistic<true>(a, b, x, s); });
    }
    store8<C>(p.dg, i, dg);
    store8<C>(p.dv, i, dv);
}

hipError_t launch_gate_grad(int c_dt, const GateGradParams& p, hipStream_t s) {
    const int64_t nb = (p.n / 8 + 255) / 256;
    const int64_t per = p.r_pad * (c_dt == DT_F32 ? 4 : 2) / 16;
    const int64_t nh = p.h != nullptr ? (p.M * per + 255) / 256 : 0;
    if (p.n % 8 != 0 || nb + nh >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    if (nb + nh == 0) return hipSuccess;
    const dim3 g((unsigned)(nb + nh));
    const bool f32 = p.dy_dt == DT_F32;
    if (c_dt == DT_F32) hipLaunchKernelGGL((gate_grad_kernel<DT_F32, DT_F32>), g, dim3(256), 0, s, p, (unsigned)nb);
    else if (c_dt == DT_F16 && f32) hipLaunchKernelGGL((gate_grad_kernel<DT_F16, DT_F32>), g, dim3(256), 0, s, p, (unsigned)nb);
    else if (c_dt == DT_F16) hipLaunchKernelGGL((gate_grad_kernel<DT_F16, DT_F16>), g, dim3(256), 0, s, p, (unsigned)nb);
    else if (f32) hipLaunchKernelGGL((gate_grad_kernel<DT_BF16, DT_F32>), g, dim3(256), 0, s, p, (unsigned)nb);
    else hipLaunchKernelGGL((gate_grad_kernel<DT_BF16, DT_BF16>), g, dim3(256), 0, s, p, (unsigned)nb);
    return hipGetLastError();
}

}  // namespace lyc
