// gated_bwd.hip -- the gated block's backward: the gradients of the two
// projections from the kept ones, and dx over both weights in one product
// (pair_tile.h, SEQ).
//
//   dg = round_c( dy * v * act'(g) )    dv = round_c( dy * act(g) )
//   dx = round_x( gh_g.down_g + gh_v.down_v + dg.W_g + dv.W_v )
#include "act.h"
#include "pair_tile.h"
#include "transpose_device.h"

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

template <int DT>
__device__ __forceinline__ uint16_t to16(float v) { return DT == DT_F16 ? f32_to_f16(v) : f32_to_bf16(v); }

// whether x, off by up to n units of 2^-24 of itself (at most as many fp32
// ulps), may lie on the other side of a border of the 16-bit type; an n that is
// no finite number says nothing of x, which then counts as undecided
template <int DT>
__device__ __forceinline__ bool near16(float x, float n) {
    if constexpr (DT == DT_BF16) {
        // borders: the low half of the bits 0x8000
        const uint32_t t = (uint32_t)__builtin_fminf(n, 32767.f) + 1u;
        return ((__builtin_bit_cast(uint32_t, x) - 0x8000u + t) & 0xFFFFu) <= 2u * t;
    } else {
        const float e = n * 0x1p-24f * __builtin_fabsf(x);   // (fp16's borders move below 2^-14)
        return !(n < __builtin_inff()) || to16<DT>(x - e) != to16<DT>(x + e);
    }
}

// (dg, dv) of one element in 64 bits, rounded to the 16-bit type once; packed
template <int DT>
__device__ __forceinline__ uint32_t grads_f64(int act, float dy, float g, float v) {
    double slope;
    const double r = act_f64(act, (double)g, &slope);
    const double x = (double)dy * (double)v * slope, y = (double)dy * r;
    const uint32_t xr = DT == DT_F16 ? f64_to_f16(x) : f64_to_bf16(x), yr = DT == DT_F16 ? f64_to_f16(y) : f64_to_bf16(y);
    return xr | (yr << 16);
}

// 8 elements per thread, the rows' shapes do not matter; bound by memory (five
// passes over M x N).  Workgroups past those copy the second half of a saved h to
// rows of its own, which the product over the tokens reads, and the factors
// transposed, which gh and dx read (a launch of their own for those cost a short
// batch 5 of 52 us).
//
// dg and dv round to 16 bits as their values in 64 bits do (the exact ones but
// for ties of dy v or dy g where act' or act / g is within 2^-53 of 1 or 1/2):
// what is built on them (gh, itself rounded, then dx and the factors' gradients)
// would carry a step taken the other way into every sum, and fp32 gradients with
// it (1e-4 of their norm).  fp32 decides all but the few in a thousand that lie within its
// error of a border; those are marked, a bit an element, and a second kernel
// evaluates them in 64 bits.  (In this one that code's registers halved the
// waves in flight: bf16 8192 x 8192 177 us with it, 113 and 32 apart.)
template <int C, int G, class T>
__global__ __launch_bounds__(256) void gate_grad_kernel(GateGradParams p, unsigned nb, unsigned nh) {
    if (blockIdx.x >= nb + nh) {
        __shared__ float lds[64][65];
        int64_t b = blockIdx.x - nb - nh;
        int k = 0;
        while (b >= transpose_tiles(p.tr[k])) b -= transpose_tiles(p.tr[k++]);
        transpose_body<T>(p.tr[k], b, (p.tr[k].rows_pad + 63) / 64, lds);
        return;
    }
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
    unsigned open = 0;   // bit e: dg or dv of element e is undecided
    float a = 1.f, b = 0.f;
    act_coeffs(p.act, a, b);
    if constexpr (C == DT_F32) {
        auto grads = [&](auto act) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float slope;
                dv[e] = dy[e] * act(g[e], &slope);
                dg[e] = dy[e] * v[e] * slope;
            }
        };
        if (p.act == ACT_GELU) grads([](float x, float* s) { float m; return act_gelu<true, true>(x, s, &m); });
        else grads([=](float x, float* s) { return act_logistic<true>(a, b, x, s); });
    } else {
        auto grads = [&](auto act) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float slope, mass, na, ns;
                const float r = act(g[e], &slope, &mass, &na, &ns);
                const float w = dy[e] * v[e];
                dg[e] = w * slope;
                dv[e] = dy[e] * r;
                // (two more units for the products with dy and value; at slope 0 the bound is infinite)
                const float nv = na + 2.f;
                const float ng = __builtin_fmaf(ns * mass, __builtin_amdgcn_rcpf(__builtin_fabsf(slope)), 2.f);
                // dy v past fp32's range, which a small slope brings back (two fp16 values never)
                const bool past = (C != DT_F16 || G != DT_F16) && __builtin_fabsf(w) == __builtin_inff();
                open |= near16<C>(dg[e], ng) || near16<C>(dv[e], nv) || past ? 1u << e : 0u;
            }
        };
        if (p.act == ACT_GELU) {
            // (below -13 exp(-g^2 / 2) nears fp32's smallest normal value)
            grads([](float x, float* s, float* m, float* na, float* ns) {
                *na = *ns = x < -13.f ? __builtin_inff() : 16.f;
                return act_gelu<true>(x, s, m);
            });
        } else {
            grads([=](float x, float* s, float* m, float* na, float* ns) {
                return act_logistic16_grad(a, b, x, s, m, na, ns);
            });
        }
    }
    store8<C>(p.dg, i, dg);
    store8<C>(p.dv, i, dv);
    if constexpr (C != DT_F32) p.open[i] = (uint8_t)open;
}

// The marked elements.  A workgroup's meet in LDS and are evaluated one a
// thread.  bf16 8192 x 8192, about 0.4% of the elements: 32 us, bound by their
// scattered reads and writes and the evaluation (a quarter of the elements a
// workgroup, whose one wave with work is then a quarter full: 44).
constexpr int FIX_N = 16384, FIX_CAP = 2048;   // elements of a workgroup, 64 a thread
template <int C, int G>
__global__ __launch_bounds__(256) void gate_fix_kernel(GateGradParams p) {
    __shared__ uint16_t queue[FIX_CAP];
    __shared__ unsigned queued;
    const int64_t first = (int64_t)blockIdx.x * FIX_N, bytes = p.n / 8, at = first / 8 + threadIdx.x * 8;
    uint64_t m = 0;
    if (at + 8 <= bytes) {
        m = *(const uint64_t*)(p.open + at);
    } else {
        for (int64_t k = at; k < bytes; ++k) m |= (uint64_t)p.open[k] << (8 * (k - at));
    }
    if (threadIdx.x == 0) queued = 0;
    __syncthreads();
    const unsigned mine = (unsigned)__builtin_popcountll(m), from = mine ? atomicAdd(&queued, mine) : 0u;
    __syncthreads();
    const unsigned all = queued;
    // (FIX_CAP a round: one but for adversarial values)
    for (unsigned base = 0; base < all; base += FIX_CAP) {
        unsigned k = from - base;   // (wraps past the end for those of earlier rounds)
        for (uint64_t o = m; o != 0; o &= o - 1, ++k)
            if (k < FIX_CAP) queue[k] = (uint16_t)(threadIdx.x * 64 + __builtin_ctzll(o));
        __syncthreads();
        const unsigned n = all - base < FIX_CAP ? all - base : FIX_CAP;
        for (unsigned q = threadIdx.x; q < n; q += 256) {
            const int64_t e = first + queue[q];
            const float dy = load_as_f32(p.dy, G, e), g = load_as_f32(p.gate, C, e), v = load_as_f32(p.value, C, e);
            const uint32_t w = grads_f64<C>(p.act, dy, g, v);
            ((uint16_t*)p.dg)[e] = (uint16_t)w;
            ((uint16_t*)p.dv)[e] = (uint16_t)(w >> 16);
        }
        __syncthreads();
    }
}

template <int C, int G>
static hipError_t run_gate_grad(const GateGradParams& p, int64_t nb, int64_t nh, int64_t nt, hipStream_t s) {
    const dim3 g((unsigned)(nb + nh + nt));
    if (p.ntr > 0 && p.tr[0].src_dt == DT_F32)
        hipLaunchKernelGGL((gate_grad_kernel<C, G, uint32_t>), g, dim3(256), 0, s, p, (unsigned)nb, (unsigned)nh);
    else
        hipLaunchKernelGGL((gate_grad_kernel<C, G, uint16_t>), g, dim3(256), 0, s, p, (unsigned)nb, (unsigned)nh);
    hipError_t e = hipGetLastError();
    if constexpr (C != DT_F32) {
        if (e == hipSuccess && nb > 0) {
            hipLaunchKernelGGL((gate_fix_kernel<C, G>), dim3((unsigned)((p.n + FIX_N - 1) / FIX_N)), dim3(256), 0, s, p);
            e = hipGetLastError();
        }
    }
    return e;
}

hipError_t launch_gate_grad(int c_dt, const GateGradParams& p, hipStream_t s) {
    const int64_t nb = (p.n / 8 + 255) / 256;
    const int64_t per = p.r_pad * (c_dt == DT_F32 ? 4 : 2) / 16;
    const int64_t nh = p.h != nullptr ? (p.M * per + 255) / 256 : 0;
    int64_t nt = 0;
    if (p.ntr < 0 || p.ntr > 4) return hipErrorInvalidValue;
    for (int i = 0; i < p.ntr; ++i) {
        if ((p.tr[i].src_dt == DT_F32) != (p.tr[0].src_dt == DT_F32)) return hipErrorInvalidValue;
        nt += transpose_tiles(p.tr[i]);
    }
    if (p.n % 8 != 0 || nb + nh + nt >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    if (nb + nh + nt == 0) return hipSuccess;
    const bool f32 = p.dy_dt == DT_F32;
    if (c_dt == DT_F32) return run_gate_grad<DT_F32, DT_F32>(p, nb, nh, nt, s);
    if (p.open == nullptr) return hipErrorInvalidValue;
    if (c_dt == DT_F16)
        return f32 ? run_gate_grad<DT_F16, DT_F32>(p, nb, nh, nt, s) : run_gate_grad<DT_F16, DT_F16>(p, nb, nh, nt, s);
    return f32 ? run_gate_grad<DT_BF16, DT_F32>(p, nb, nh, nt, s) : run_gate_grad<DT_BF16, DT_BF16>(p, nb, nh, nt, s);
}

}  // namespace lyc
