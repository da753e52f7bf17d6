// ortho.hip -- Newton-Schulz orthogonalization of an update G [R][C]:
//
//   X0 = G / (|G|_F + eps);   X <- a X + (b A + c A^2) X,  A = X X^T
//
// with A over the short side n (m the long one; a tall G is taken as the
// transpose of a wide one, as stored: no transposed copy is made).  Each step
// is three products, A = X X^T, A^2 with P = a I + b A + c A^2 in its
// epilogue, and X <- P X.
//
// Precision.  A step amplifies small singular values by a (3.4 by default),
// rounding errors of X with them, so 16-bit operands would leave errors of a
// percent.  Operands are split into 16-bit pieces and their products summed in
// fp32 by 16-bit MFMAs:
//   16-bit G: two fp16 pieces (22 bits), 3 of the 4 products; the matrices are
//     scaled by powers of two that the coefficients' bounds keep inside fp16;
//   fp32 G: three bf16 pieces (24 bits), 6 of the 9 products.
#include <algorithm>
#include <cmath>

#include "gemm_tile.h"
#include "kernels.h"
#include "lyc_device.h"
#include "ortho.h"

namespace lyc {

// ---- pieces ---------------------------------------------------------------------

// NP = 2: fp16 pieces, NP = 3: bf16 pieces
template <int NP>
struct Pieces {
    using CT = CF16;
    static __device__ __forceinline__ void split(float v, uint16_t (&o)[2]) {
        o[0] = f32_to_f16(v);
        o[1] = f32_to_f16(v - f16_to_f32(o[0]));
    }
    static __device__ __forceinline__ float join(const uint16_t (&o)[2]) { return f16_to_f32(o[0]) + f16_to_f32(o[1]); }
};
template <>
struct Pieces<3> {
    using CT = CBF16;
    static __device__ __forceinline__ void split(float v, uint16_t (&o)[3]) {
        o[0] = f32_to_bf16(v);
        const float r = v - bf16_to_f32(o[0]);
        o[1] = f32_to_bf16(r);
        o[2] = f32_to_bf16(r - bf16_to_f32(o[1]));
    }
    static __device__ __forceinline__ float join(const uint16_t (&o)[3]) {
        return bf16_to_f32(o[0]) + (bf16_to_f32(o[1]) + bf16_to_f32(o[2]));
    }
};

// A matrix as pieces: [rows][ld] per piece, ld a multiple of 8, zero past cols
struct Planes {
    uint16_t* p;
    int64_t ld, stride;   // stride: elements between pieces
};

// ---- the norm and the first split --------------------------------------------------

constexpr int NORM_WGS = 256;

__global__ __launch_bounds__(256) void ns_norm_kernel(const void* g, int dt, int64_t n, double* part) {
    __shared__ double red[4];
    const int tid = threadIdx.x;
    double s = 0;
    for (int64_t i = (int64_t)blockIdx.x * 256 + tid; i < n; i += (int64_t)NORM_WGS * 256) {
        const double v = (double)load_as_f32(g, dt, i);
        s += v * v;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if ((tid & 63) == 0) red[tid >> 6] = s;
    __syncthreads();
    if (tid == 0) part[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// 1 / (|G|_F + eps) from the partial sums, the same in every thread
__device__ __forceinline__ double ns_inverse_norm(const double* part, double eps) {
    const int lane = threadIdx.x & 63;
    double s = 0;
#pragma unroll
    for (int i = 0; i < NORM_WGS / 64; ++i) s += part[i * 64 + lane];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    return 1.0 / (__builtin_sqrt(s) + eps);
}

template <int NP>
__global__ __launch_bounds__(256) void ns_split_kernel(const void* g, int dt, int64_t rows, int64_t cols, Planes x,
                                                       const double* part, double eps, float scale) {
    const double inv = ns_inverse_norm(part, eps);
    const int64_t total = rows * x.ld;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / x.ld, c = i - r * x.ld;
        const float v = c < cols ? (float)((double)load_as_f32(g, dt, r * cols + c) * inv) * scale : 0.f;
        uint16_t o[NP];
        Pieces<NP>::split(v, o);
#pragma unroll
        for (int k = 0; k < NP; ++k) x.p[k * x.stride + i] = o[k];
    }
}

// ---- the products ----------------------------------------------------------------------

enum { NS_SPLIT = 0, NS_POLY = 1, NS_OUT = 2 };

// out(j, i) = finish( alpha * sum_k U(i, k) V(j, k) ), i < I, j < J, k < K.
// Rows-as-stored form: u [I][ld], v [J][ld], k consecutive.  Transposed form:
// u [K][ld], v [K][ld].
//   NS_SPLIT: v' = sum                      into pieces, times `scale`
//   NS_POLY:  v' = a delta_ij + b A + c sum into pieces, times `scale`; A from `old`
//   NS_OUT:   v' into out [J][I] of dtype dt
struct NsParams {
    Planes u, v, o, old;
    int64_t I, J, K;
    float alpha, scale;
    float a, b, c, old_inv;
    int mode;
    void* out;
    int dt;
    int ksplit;
    float* partial;   // [ksplit][J][I rounded up to 4] when ksplit > 1
};

template <int NP>
__device__ __forceinline__ float ns_value(const NsParams& p, float sum, int64_t j, int64_t i) {
    float v = sum * p.alpha;
    if (p.mode == NS_POLY) {
        uint16_t w[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) w[k] = p.old.p[k * p.old.stride + j * p.old.ld + i];
        v = p.c * v + p.b * (Pieces<NP>::join(w) * p.old_inv);
        if (i == j) v += p.a;
    }
    return v;
}

// four consecutive i of row j (j < J; i past the row's end masked)
template <int NP>
__device__ __forceinline__ void ns_finish4(const NsParams& p, f32x4 s, int64_t j, int64_t i) {
    if (p.mode == NS_OUT) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i + e >= p.I) continue;
            const float v = ns_value<NP>(p, s[e], j, i + e);
            const int64_t at = j * p.I + i + e;
            if (p.dt == DT_F32) ((float*)p.out)[at] = v;
            else ((uint16_t*)p.out)[at] = p.dt == DT_F16 ? f32_to_f16(v) : f32_to_bf16(v);
        }
        return;
    }
    if (i >= p.o.ld) return;   // (ld a multiple of 8: all four or none)
    uint16_t o[4][NP];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float v = i + e < p.I ? ns_value<NP>(p, s[e], j, i + e) : 0.f;
        Pieces<NP>::split(v * p.scale, o[e]);
    }
#pragma unroll
    for (int k = 0; k < NP; ++k)
        *(i32x2*)(p.o.p + k * p.o.stride + j * p.o.ld + i) =
            i32x2{(int)((uint32_t)o[0][k] | (uint32_t)o[1][k] << 16), (int)((uint32_t)o[2][k] | (uint32_t)o[3][k] << 16)};
}

// One side's rows of a K step (32 k) in LDS, and its loads.
//   as stored: ROWS rows of 64 bytes, 16-byte chunk c of row r at slot
//     c ^ ((r / 2) % 4);
//   transposed: 32 rows of ROWS * 2 bytes, the layout of frag_t.
template <int ROWS, int NW, bool TR>
struct NsSide {
    static constexpr int Q = ROWS / 16 / NW;   // 1 KiB wave loads per wave and piece
    static_assert(Q * 16 * NW == ROWS, "loader split");
    static constexpr int BYTES = ROWS * 64;
    static constexpr int CPR = ROWS / 8, KRB = 64 / CPR;
    uint32_t off, step_q;
    const char* base;
    uint32_t row_bytes;
    int64_t k_rows;
    int rows;
    __device__ __forceinline__ void init(const Planes& m, int64_t r0, int64_t nrows, int64_t K, int wave, int lane) {
        row_bytes = (uint32_t)(m.ld * 2);
        if constexpr (TR) {
            const int r = wave * KRB + lane / CPR;
            const int64_t col = r0 + 8 * ((lane % CPR) ^ tswz<CPR>(r));
            off = col < m.ld ? (uint32_t)((r * m.ld + col) * 2) : OOB;
            step_q = (uint32_t)(NW * KRB * m.ld * 2);
            base = (const char*)m.p;
            k_rows = K;
        } else {
            const int r = wave * 16 + lane / 4;
            off = (uint32_t)r * row_bytes + (uint32_t)(((lane & 3) ^ ((r >> 1) & 3)) << 4);
            step_q = (uint32_t)(NW * 16) * row_bytes;
            base = (const char*)m.p + r0 * row_bytes;
            rows = (int)(nrows - r0 < ROWS ? nrows - r0 : ROWS);
        }
    }
    // loads of K step s of one piece (pointer offset po) into LDS at dst
    __device__ __forceinline__ void issue(char* dst, int64_t po, int64_t s, bool on, int wave, int lane) const {
        if constexpr (TR) {
            const int64_t left = k_rows - s * 32;
            const uint32_t nrow = on && left > 0 ? (uint32_t)(left < 32 ? left : 32) : 0u;
            const auto rs = make_rsrc(base + po + s * 32 * (int64_t)row_bytes, nrow * row_bytes);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                auto* d = (__attribute__((address_space(3))) void*)(dst + (wave + q * NW) * 1024);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, d, 16, off == OOB ? OOB : off + (uint32_t)q * step_q, 0, 0, 0);
            }
        } else {
            const auto rs = make_rsrc(base + po, on ? (uint32_t)rows * row_bytes : 0u);
            const uint32_t kb = (uint32_t)(s * 64);
            const int r = wave * 16 + lane / 4;
            const bool ok = kb + (uint32_t)(((lane & 3) ^ ((r >> 1) & 3)) << 4) < row_bytes;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                auto* d = (__attribute__((address_space(3))) void*)(dst + (wave + q * NW) * 1024);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, d, 16, ok ? off + (uint32_t)q * step_q : OOB, (int)kb, 0, 0);
            }
        }
    }
    static __device__ __forceinline__ i32x4 frag(const char* tile, int r0, int lane) {
        if constexpr (TR) {
            return frag_t<ROWS>(tile, 0, r0, lane);
        } else {
            const int r = r0 + (lane & 15);
            return *(const i32x4*)(tile + r * 64 + (((lane >> 4) ^ ((r >> 1) & 3)) << 4));
        }
    }
};

// T x T output tile per workgroup of 4 waves (2 x 2), NS stages of one K step
// (32 k of every piece of both sides).
template <int NP, bool TR, int T, int NS>
__global__ __launch_bounds__(256, NP == 2 ? 2 : 1) void ns_gemm_kernel(NsParams p, int tiles_i, int tiles_j) {
    constexpr int NW = 4, W = T / 2, F = W / 16;
    using Side = NsSide<T, NW, TR>;
    constexpr int STAGE = 2 * NP * Side::BYTES, Q = 2 * NP * Side::Q;
    static_assert(NS * STAGE <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(16))) char smem[NS * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave & 1, wj = wave >> 1;
    int ti, tj;
    tile_coords(blockIdx.x, gridDim.x, tiles_i, tiles_j, 4, ti, tj);
    const int64_t i0 = (int64_t)ti * T, j0 = (int64_t)tj * T;
    Side su, sv;
    su.init(p.u, i0, p.I, p.K, wave, lane);
    sv.init(p.v, j0, p.J, p.K, wave, lane);
    const int64_t steps = (p.K + 31) / 32, per = (steps + p.ksplit - 1) / p.ksplit;
    const int64_t s0 = (int64_t)blockIdx.y * per;
    const int KT = (int)(steps - s0 < per ? (steps - s0 > 0 ? steps - s0 : 0) : per);

    auto issue = [&](int kt) {
        char* st = smem + (kt % NS) * STAGE;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            su.issue(st + k * Side::BYTES, k * p.u.stride * 2, s0 + kt, kt < KT, wave, lane);
            sv.issue(st + (NP + k) * Side::BYTES, k * p.v.stride * 2, s0 + kt, kt < KT, wave, lane);
        }
    };
    f32x4 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) issue(s);
    for (int kt = 0; kt < KT; ++kt) {
        wait_vm<(NS - 2) * Q>();
        lds_barrier();
        issue(kt + NS - 1);
        const char* st = smem + (kt % NS) * STAGE;
        i32x4 b[NP][F];
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int j = 0; j < F; ++j) b[k][j] = Side::frag(st + (NP + k) * Side::BYTES, wj * W + j * 16, lane);
#pragma unroll
        for (int i = 0; i < F; ++i) {
            i32x4 a[NP];
#pragma unroll
            for (int k = 0; k < NP; ++k) a[k] = Side::frag(st + k * Side::BYTES, wi * W + i * 16, lane);
            // piece products whose orders add up to at most NP - 1
#pragma unroll
            for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                for (int k = 0; k <= o; ++k)
#pragma unroll
                    for (int j = 0; j < F; ++j) acc[i][j] = Pieces<NP>::CT::step(a[k], b[o - k][j], acc[i][j]);
        }
    }
    wait_vm<0>();
    const int g = lane >> 4, r = lane & 15;
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int64_t oi = i0 + wi * W + i * 16 + 4 * g;
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int64_t oj = j0 + wj * W + j * 16 + r;
            if (oj >= p.J) continue;
            if (p.ksplit > 1) {
                const int64_t ldp = (p.I + 3) & ~(int64_t)3;
                if (oi < ldp) *(f32x4*)(p.partial + ((int64_t)blockIdx.y * p.J + oj) * ldp + oi) = acc[i][j];
            } else {
                ns_finish4<NP>(p, acc[i][j], oj, oi);
            }
        }
    }
}

// sums of the K splits in split order, then the same finish
template <int NP>
__global__ __launch_bounds__(256) void ns_reduce_kernel(NsParams p) {
    const int64_t ldp = (p.I + 3) & ~(int64_t)3;
    // (pieces: up to the padded row end, whose last four are zeros)
    const int64_t q = (p.mode == NS_OUT ? ldp : p.o.ld) / 4;
    const int64_t total = p.J * q;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t j = t / q, i = (t - j * q) * 4;
        f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
        if (i < ldp)
            for (int k = 0; k < p.ksplit; ++k) s += *(const f32x4*)(p.partial + ((int64_t)k * p.J + j) * ldp + i);
        ns_finish4<NP>(p, s, j, i);
    }
}

// ---- host ----------------------------------------------------------------------------------

static int64_t up8(int64_t v) { return (v + 7) & ~(int64_t)7; }
static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// tile and K split of an I x J product over K: 128 x 128 tiles where they fill
// half the device, else 64 x 64; a K split while workgroups are fewer than the
// CUs, at least 4 steps of 32 each
static void ns_plan(int64_t I, int64_t J, int64_t K, int* tile, int* ksplit) {
    const int64_t cus = device_rates().cus;
    const int64_t big = ((I + 127) / 128) * ((J + 127) / 128);
    *tile = big >= cus / 2 ? 128 : 64;
    const int64_t t = *tile, tiles = ((I + t - 1) / t) * ((J + t - 1) / t);
    const int64_t steps = (K + 31) / 32;
    int64_t ks = tiles > 0 ? cus / tiles : 1;
    ks = std::min<int64_t>(ks, steps / 4);
    ks = std::min<int64_t>(ks, 64);
    *ksplit = ks > 1 ? (int)ks : 1;
}

struct NsLayout {
    size_t norm, x[2], A, P, partial, total;
    int64_t ldx, ldn, rows;
};
static NsLayout ns_layout(int64_t R, int64_t C, int dt) {
    const size_t np = dt == DT_F32 ? 3 : 2;
    const int64_t n = std::min(R, C), m = std::max(R, C);
    NsLayout L{};
    L.rows = R;
    L.ldx = up8(C);
    L.ldn = up8(n);
    size_t off = 0;
    auto take = [&](size_t& at, size_t bytes) { at = off; off = up256(off + bytes); };
    take(L.norm, NORM_WGS * sizeof(double));
    for (int i = 0; i < 2; ++i) take(L.x[i], np * (size_t)(R * L.ldx) * 2);
    take(L.A, np * (size_t)(n * L.ldn) * 2);
    take(L.P, np * (size_t)(n * L.ldn) * 2);
    size_t part = 0;
    int t, ks;
    ns_plan(n, n, m, &t, &ks);
    if (ks > 1) part = std::max(part, (size_t)ks * (size_t)(n * ((n + 3) & ~(int64_t)3)) * 4);
    ns_plan(n, n, n, &t, &ks);
    if (ks > 1) part = std::max(part, (size_t)ks * (size_t)(n * ((n + 3) & ~(int64_t)3)) * 4);
    ns_plan(C, R, n, &t, &ks);
    if (ks > 1) part = std::max(part, (size_t)ks * (size_t)(R * ((C + 3) & ~(int64_t)3)) * 4);
    take(L.partial, part);
    L.total = off;
    return L;
}
size_t ortho_workspace(int64_t R, int64_t C, int dt) { return R > 0 && C > 0 ? ns_layout(R, C, dt).total : 0; }

template <int NP, bool TR>
static hipError_t ns_product(NsParams p, hipStream_t s) {
    int t;
    ns_plan(p.I, p.J, p.K, &t, &p.ksplit);
    const int ti = (int)((p.I + t - 1) / t), tj = (int)((p.J + t - 1) / t);
    const dim3 grid((unsigned)(ti * tj), (unsigned)p.ksplit);
    if (t == 128) hipLaunchKernelGGL((ns_gemm_kernel<NP, TR, 128, 2>), grid, dim3(256), 0, s, p, ti, tj);
    else hipLaunchKernelGGL((ns_gemm_kernel<NP, TR, 64, 3>), grid, dim3(256), 0, s, p, ti, tj);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.ksplit > 1) {
        const int64_t q = p.J * ((p.mode == NS_OUT ? (p.I + 3) / 4 : p.o.ld / 4));
        hipLaunchKernelGGL(ns_reduce_kernel<NP>, dim3((unsigned)std::min<int64_t>((q + 255) / 256, 4096)), dim3(256), 0, s, p);
        e = hipGetLastError();
    }
    return e;
}

template <int NP>
static hipError_t ns_direct(const OrthoParams& p, hipStream_t s) {
    const NsLayout L = ns_layout(p.R, p.C, p.dt);
    const bool tall = p.R > p.C;
    const int64_t n = std::min(p.R, p.C), m = std::max(p.R, p.C);
    char* W = p.ws;
    double* part = (double*)(W + L.norm);
    Planes x[2], A, P;
    for (int i = 0; i < 2; ++i) x[i] = Planes{(uint16_t*)(W + L.x[i]), L.ldx, p.R * L.ldx};
    A = Planes{(uint16_t*)(W + L.A), L.ldn, n * L.ldn};
    P = Planes{(uint16_t*)(W + L.P), L.ldn, n * L.ldn};

    // power-of-two scales that keep every element inside fp16: elements are at
    // most the spectral norm, which the scalar map s -> s p(s^2) bounds
    // (A's eigenvalues lie in [0, top])
    double top = 1.0, sx = 1.0, pmax = 0.0;
    double topx = 1.0;
    for (int k = 0; k < p.steps; ++k) {
        double next = 0.0;
        for (int i = 0; i <= 512; ++i) {
            const double l = top * i / 512.0, q = p.a + l * (p.b + l * p.c);
            pmax = std::max(pmax, std::fabs(q));
            next = std::max(next, l * q * q);
        }
        next *= 1.02;   // between the sampled points, and the products' rounding
        if (!(next < 1e30)) next = 1e30;
        top = next;
        topx = std::max(topx, top);
    }
    auto pow2_under = [](double bound) {   // the largest power of two with scale * bound <= 2^15
        return std::ldexp(1.0, std::min(15, (int)std::floor(15.0 - std::log2(std::max(bound, 1e-30)))));
    };
    double sa = 1.0, sp = 1.0;
    if (NP == 2) {
        sx = pow2_under(std::sqrt(topx));
        sa = pow2_under(topx);
        sp = pow2_under(std::max(pmax, 1e-30));
    }

    hipLaunchKernelGGL(ns_norm_kernel, dim3(NORM_WGS), dim3(256), 0, s, p.g, p.dt, p.R * p.C, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t wgs = std::min<int64_t>((p.R * L.ldx + 255) / 256, 2048);
    hipLaunchKernelGGL(ns_split_kernel<NP>, dim3((unsigned)wgs), dim3(256), 0, s, p.g, p.dt, p.R, p.C, x[0], part, p.eps,
                       (float)sx);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    for (int k = 0; k < p.steps; ++k) {
        const Planes& cur = x[k & 1];
        NsParams q{};
        q.partial = (float*)(W + L.partial);
        // A = X X^T
        q.u = q.v = cur;
        q.o = A;
        q.I = q.J = n;
        q.K = m;
        q.alpha = (float)(1.0 / (sx * sx));
        q.scale = (float)sa;
        q.mode = NS_SPLIT;
        e = tall ? ns_product<NP, true>(q, s) : ns_product<NP, false>(q, s);
        if (e != hipSuccess) return e;
        // P = a I + b A + c A A
        q.u = q.v = q.old = A;
        q.o = P;
        q.K = n;
        q.alpha = (float)(1.0 / (sa * sa));
        q.old_inv = (float)(1.0 / sa);
        q.scale = (float)sp;
        q.a = (float)p.a;
        q.b = (float)p.b;
        q.c = (float)p.c;
        q.mode = NS_POLY;
        if ((e = ns_product<NP, false>(q, s)) != hipSuccess) return e;
        // X <- P X (stored [R][C]: i runs over C, j over R)
        q.alpha = (float)(1.0 / (sx * sp));
        q.scale = (float)sx;
        q.o = x[(k + 1) & 1];
        q.I = p.C;
        q.J = p.R;
        q.K = n;
        q.mode = k + 1 < p.steps ? NS_SPLIT : NS_OUT;
        q.out = p.out;
        q.dt = p.dt;
        if (tall) {
            q.u = P;
            q.v = cur;
            e = ns_product<NP, false>(q, s);
        } else {
            q.u = cur;
            q.v = P;
            e = ns_product<NP, true>(q, s);
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_ortho(const OrthoParams& p, hipStream_t s) {
    if (p.R <= 0 || p.C <= 0) return hipSuccess;
    return p.dt == DT_F32 ? ns_direct<3>(p, s) : ns_direct<2>(p, s);
}

}  // namespace lyc
