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
//   16-bit G: two fp16 pieces (22 bits), 3 of the 4 products;
//   fp32 G: three bf16 pieces (24 bits), 6 of the 9 products.  They have fp32's
//     range, so a 16-bit G whose coefficients leave X's size unknown by too
//     much (ns_loose) takes them too.
// Every matrix is held times a power of two that puts its largest possible
// element near the top of fp16 (near 1 for bf16), step by step: the bits are
// there whatever the size of G beside eps and wherever the coefficients take X.
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

// c[i][j] += a[i] . b[j] over the piece products whose orders add up to at
// most NP - 1, small ones first; consecutive MFMAs go to different tiles
template <int NP, int I, int J>
__device__ __forceinline__ void piece_mma(const i32x4 (&a)[I][NP], const i32x4 (&b)[J][NP], f32x4 (&c)[I][J]) {
#pragma unroll
    for (int o = NP - 1; o >= 0; --o)
#pragma unroll
        for (int k = 0; k <= o; ++k)
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int j = 0; j < J; ++j) c[i][j] = Pieces<NP>::CT::step(a[i][k], b[j][o - k], c[i][j]);
}

// 2^e as two factors, for an e past fp32's exponents (an ldexp takes as long as
// four products)
struct Pow2 {
    float a, b;
    static __device__ __forceinline__ float one(int e) {
        e = e < -126 ? -126 : e > 126 ? 126 : e;
        return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
    }
    explicit __device__ __forceinline__ Pow2(int e) : a(one(e / 2)), b(one(e - e / 2)) {}
    __device__ __forceinline__ float operator()(float v) const { return v * a * b; }
};

// A matrix as pieces: [rows][ld] per piece, ld a multiple of 8, zero past cols
struct Planes {
    uint16_t* p;
    int64_t ld, stride;   // stride: elements between pieces
};

// ---- the norm and the first split --------------------------------------------------

constexpr int NORM_WGS = 512;

// 16 elements from `at` of the flat matrix of n elements as fp32 (zeros past
// it): 16-byte loads where vec (the matrix 16-byte aligned, 16 elements left)
__device__ __forceinline__ void load16_f32(const void* g, int dt, int64_t at, int64_t n, bool vec, float (&v)[16]) {
    if (vec && at + 16 <= n) {
        i32x4 w[4];
        const i32x4* src = (const i32x4*)((const char*)g + at * (dt == DT_F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = src[i];
        if (dt == DT_F32) {
#pragma unroll
            for (int i = 2; i < 4; ++i) w[i] = src[i];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __builtin_bit_cast(float, (uint32_t)w[e >> 2][e & 3]);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t u = (uint32_t)w[e >> 3][(e >> 1) & 3];
                const uint16_t h = (uint16_t)((e & 1) ? u >> 16 : u);
                v[e] = dt == DT_F16 ? f16_to_f32(h) : bf16_to_f32(h);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = at + e < n ? load_as_f32(g, dt, at + e) : 0.f;
    }
}

__global__ __launch_bounds__(256) void ns_norm_kernel(const void* g, int dt, int64_t n, int vec, double* part) {
    __shared__ double red[4];
    const int tid = threadIdx.x;
    double s = 0;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + tid) * 16; i < n; i += (int64_t)NORM_WGS * 256 * 16) {
        float v[16];
        load16_f32(g, dt, i, n, vec, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) s = __builtin_fma((double)v[e], (double)v[e], s);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if ((tid & 63) == 0) red[tid >> 6] = s;
    __syncthreads();
    if (tid == 0) part[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// 1 / (|G|_F + eps); a zero G with eps = 0 stays zero
__device__ __forceinline__ double ns_inverse(double norm, double eps) {
    const double d = norm + eps;
    return d == 0.0 ? 0.0 : 1.0 / d;
}

// |G|_F from the partial sums, the same in every thread
__device__ __forceinline__ double ns_norm(const double* part) {
    const int lane = threadIdx.x & 63;
    double s = 0;
#pragma unroll
    for (int i = 0; i < NORM_WGS / 64; ++i) s += part[i * 64 + lane];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    return __builtin_sqrt(s);
}

// The powers of two of a dense update's products, five a step: A = ldexp of
// the sum of X X^T; P's of c A A, of b A and of a; ldexp of the sum of P X (into
// the next X, or the result itself after the last step).
constexpr int NS_EXPS = 5;

// A matrix of spectral norm up to `bound` (its elements are at most that) is
// held times 2^ns_exponent: below 2^15 in fp16 pieces, below 1 in bf16 ones.
template <int NP>
__host__ __device__ inline int ns_exponent(double bound) {
    if (!(bound > 0.0 && bound < 1e300)) return 0;
    int e;
    frexp(bound, &e);   // bound < 2^e
    return (NP == 2 ? 15 : 0) - e;
}

// What a step does to eigenvalues of A in [0, top]: the largest |p|, |l p| and
// next eigenvalue l p^2, at the ends or where the derivative's quadratic
// u + v l + w l^2 vanishes.
struct NsBounds {
    double p, lp, next;
};
__host__ __device__ inline NsBounds ns_bounds(double a, double b, double c, double top) {
    double m[3];
    for (int i = 0; i < 3; ++i) {
        const double u = i == 0 ? b : a;
        const double v = i == 0 ? 2 * c : i == 1 ? 2 * b : 3 * b;
        const double w = i == 0 ? 0.0 : i == 1 ? 3 * c : 5 * c;
        auto f = [&](double l) {
            const double p = a + l * (b + l * c);
            return fabs(i == 0 ? p : i == 1 ? l * p : l * p * p);   // (where p vanishes so does l p^2)
        };
        double t = fmax(f(0.0), f(top));
        auto at = [&](double l) { if (l > 0.0 && l < top) t = fmax(t, f(l)); };
        const double d = v * v - 4 * u * w;
        if (w == 0.0) {
            if (v != 0.0) at(-u / v);
        } else if (d >= 0.0) {
            at((-v - sqrt(d)) / (2 * w));
            at((-v + sqrt(d)) / (2 * w));
        }
        t *= 1.01;   // the products' rounding
        m[i] = t < 1e290 ? t : 1e290;
    }
    return NsBounds{m[0], m[1], m[2]};
}

// the table, from a bound of |X0|_F
template <int NP, class T>
__host__ __device__ void ns_exponents(T* e, int steps, double a, double b, double c, double theta) {
    double top = theta * theta;
    int ex = ns_exponent<NP>(theta);
    for (int k = 0; k < steps; ++k) {
        const NsBounds n = ns_bounds(a, b, c, top);
        const int ea = ns_exponent<NP>(top), ep = ns_exponent<NP>(n.p), en = ns_exponent<NP>(sqrt(n.next));
        e[0] = (T)(ea - 2 * ex);
        e[1] = (T)(ep - 2 * ea);
        e[2] = (T)(ep - ea);
        e[3] = (T)ep;
        e[4] = (T)((k + 1 < steps ? en : 0) - ex - ep);
        e += NS_EXPS;
        top = n.next;
        ex = en;
    }
}

// x = pieces of g / (|g| + eps), 8 columns a thread (rows padded to 8 columns
// with zeros), and the table of the powers of two of what follows: the host's
// where |X0| > 1/2, which is where |G| > eps; one lane makes another from |X0|
// itself (8 us for five steps).
struct SplitParams {
    const void* g;
    int dt;
    int64_t rows, cols;
    Planes x;
    const double* part;
    int* exps;   // [steps][NS_EXPS]
    int steps;
    double a, b, c, eps;
    short usual[ORTHO_MAX_STEPS * NS_EXPS];   // the table for |X0| = 1
};
template <int NP>
__global__ __launch_bounds__(256) void ns_split_kernel(SplitParams p) {
    const void* g = p.g;
    const int dt = p.dt;
    const int64_t rows = p.rows, cols = p.cols;
    const Planes x = p.x;
    // (the whole factor in 64 bits: a norm near fp32's ends has no fp32 reciprocal)
    const double norm = ns_norm(p.part), inv = ns_inverse(norm, p.eps);
    const double theta = norm * inv;
    const bool usual = theta > 0.5;
    const double f = ldexp(inv, ns_exponent<NP>(usual ? 1.0 : theta));
    if (blockIdx.x == 0) {
        if (usual) {
            if ((int)threadIdx.x < p.steps * NS_EXPS) p.exps[threadIdx.x] = p.usual[threadIdx.x];
        } else if (threadIdx.x == 0) {
            ns_exponents<NP>(p.exps, p.steps, p.a, p.b, p.c, theta);
        }
    }
    const int64_t q = x.ld / 8, total = rows * q;
    const bool vec = cols % 8 == 0 && ((uintptr_t)g & 15) == 0;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t r = t / q, c = (t - r * q) * 8;
        uint32_t raw[8];
        if (vec) {
            const char* src = (const char*)g + (r * cols + c) * (dt == DT_F32 ? 4 : 2);
            const i32x4 a = *(const i32x4*)src;
            if (dt == DT_F32) {
                const i32x4 b = *(const i32x4*)(src + 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) { raw[e] = (uint32_t)a[e]; raw[4 + e] = (uint32_t)b[e]; }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) raw[e] = (uint32_t)a[e >> 1] >> (16 * (e & 1)) & 0xFFFFu;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t at = r * cols + (c + e < cols ? c + e : cols - 1);
                const uint32_t w = dt == DT_F32 ? ((const uint32_t*)g)[at] : ((const uint16_t*)g)[at];
                raw[e] = c + e < cols ? w : 0u;
            }
        }
        uint16_t o[8][NP];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = dt == DT_F32 ? __builtin_bit_cast(float, raw[e])
                                         : (dt == DT_F16 ? f16_to_f32((uint16_t)raw[e]) : bf16_to_f32((uint16_t)raw[e]));
            Pieces<NP>::split((float)((double)v * f), o[e]);
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            i32x4 w;
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] = (int)((uint32_t)o[2 * u][k] | (uint32_t)o[2 * u + 1][k] << 16);
            *(i32x4*)(x.p + k * x.stride + r * x.ld + c) = w;
        }
    }
}

// ---- the products ----------------------------------------------------------------------

enum { NS_SPLIT = 0, NS_POLY = 1, NS_OUT = 2 };

// out(j, i) = finish( s = sum_k U(i, k) V(j, k) ), i < I, j < J, k < K.
// Each of u and v rows-as-stored ([I or J][ld], k consecutive) or transposed
// ([K][ld]); e: this product's powers of two in the table.
//   NS_SPLIT: 2^e0 s                                  into pieces
//   NS_POLY:  2^e2 a delta_ij + 2^e1 b A + 2^e0 c s   into pieces; A from `old`
//   NS_OUT:   2^e0 s                                  into out [J][I] of dtype dt
struct NsParams {
    Planes u, v, o, old;
    int64_t I, J, K;
    const int* e;
    float a, b, c;
    int mode;
    void* out;
    int dt;
    int sym;          // out is symmetric: only tiles that reach i >= j, mirrored by ns_sym_reduce_kernel
    int ksplit;
    float* partial;   // [ksplit][J][I rounded up to 4] when ksplit > 1 or sym
};

// a product's entries of the table, read at the kernel's start (at its end the
// load would be waited for; left to the compiler, bf16 256 x 4096 took 199.5 us,
// not 197.5)
struct NsExps {
    int e0, e1, e2;
    explicit __device__ __forceinline__ NsExps(const NsParams& p)
        : e0(__builtin_amdgcn_readfirstlane(p.e[0])), e1(__builtin_amdgcn_readfirstlane(p.e[1])),
          e2(__builtin_amdgcn_readfirstlane(p.e[2])) {}
};

// the finished values of four consecutive i of row j from their sums (i a
// multiple of 4 inside a row of pieces; zeros past I)
template <int NP>
__device__ __forceinline__ void ns_values4(const NsParams& p, const NsExps& x, f32x4 s, int64_t j, int64_t i,
                                           float (&v)[4]) {
    const Pow2 f0(x.e0);
    if (p.mode == NS_POLY) {
        const Pow2 f1(x.e1), f2(x.e2);
        i32x2 w[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) w[k] = *(const i32x2*)(p.old.p + k * p.old.stride + j * p.old.ld + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint16_t u[NP];
#pragma unroll
            for (int k = 0; k < NP; ++k) u[k] = (uint16_t)((uint32_t)w[k][e >> 1] >> (e & 1) * 16);
            v[e] = f0(p.c * s[e]) + f1(p.b * Pieces<NP>::join(u));
            if (i + e == j) v[e] += f2(p.a);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = f0(s[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < p.I ? v[e] : 0.f;
}

template <int NP>
__device__ __forceinline__ void ns_store4(const NsParams& p, const float (&v)[4], int64_t j, int64_t i) {
    uint16_t o[4][NP];
#pragma unroll
    for (int e = 0; e < 4; ++e) Pieces<NP>::split(v[e], o[e]);
#pragma unroll
    for (int k = 0; k < NP; ++k)
        *(i32x2*)(p.o.p + k * p.o.stride + j * p.o.ld + i) =
            i32x2{(int)((uint32_t)o[0][k] | (uint32_t)o[1][k] << 16), (int)((uint32_t)o[2][k] | (uint32_t)o[3][k] << 16)};
}

// four consecutive i of row j (j < J; i past the row's end masked)
template <int NP>
__device__ __forceinline__ void ns_finish4(const NsParams& p, const NsExps& x, f32x4 s, int64_t j, int64_t i) {
    if (p.mode == NS_OUT) {
        const Pow2 f0(x.e0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i + e >= p.I) continue;
            const float v = f0(s[e]);
            const int64_t at = j * p.I + i + e;
            if (p.dt == DT_F32) ((float*)p.out)[at] = v;
            else ((uint16_t*)p.out)[at] = p.dt == DT_F16 ? f32_to_f16(v) : f32_to_bf16(v);
        }
        return;
    }
    if (i >= p.o.ld) return;   // (ld a multiple of 8: all four or none)
    float v[4];
    ns_values4<NP>(p, x, s, j, i, v);
    ns_store4<NP>(p, v, j, i);
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

// tiles of tile row ti that hold an element with i >= j
__host__ __device__ __forceinline__ int sym_tiles(int ti, int TI, int TJ, int tiles_j) {
    const int c = (ti * TI + TI - 1) / TJ + 1;
    return c < tiles_j ? c : tiles_j;
}

// TI x TJ output tile per workgroup of WVI x WVJ waves, NS stages of one K
// step (32 k of every piece of both sides).
template <int NP, bool TRU, bool TRV, int TI, int TJ, int WVI, int WVJ, int NS>
__global__ __launch_bounds__(64 * WVI * WVJ, 1) void ns_gemm_kernel(NsParams p, int tiles_i, int tiles_j) {
    constexpr int NW = WVI * WVJ, WI = TI / WVI, WJ = TJ / WVJ, FI = WI / 16, FJ = WJ / 16;
    using SideU = NsSide<TI, NW, TRU>;
    using SideV = NsSide<TJ, NW, TRV>;
    constexpr int STAGE = NP * (SideU::BYTES + SideV::BYTES), Q = NP * (SideU::Q + SideV::Q);
    static_assert(NS * STAGE <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(16))) char smem[NS * STAGE];
    const NsExps exps(p);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave % WVI, wj = wave / WVI;
    int ti, tj;
    if (p.sym) {
        // the first tj of row ti are wanted; each XCD takes a run of the list
        const int n = gridDim.x, per = n >> 3, rem = n & 7, xcd = blockIdx.x & 7;
        tj = xcd * per + (xcd < rem ? xcd : rem) + ((int)blockIdx.x >> 3);
        for (ti = 0;; ++ti) {
            const int c = sym_tiles(ti, TI, TJ, tiles_j);
            if (tj < c) break;
            tj -= c;
        }
    } else {
        tile_coords(blockIdx.x, gridDim.x, tiles_i, tiles_j, 4, ti, tj);
    }
    const int64_t i0 = (int64_t)ti * TI, j0 = (int64_t)tj * TJ;
    SideU su;
    SideV sv;
    su.init(p.u, i0, p.I, p.K, wave, lane);
    sv.init(p.v, j0, p.J, p.K, wave, lane);
    const int64_t steps = (p.K + 31) / 32, per = (steps + p.ksplit - 1) / p.ksplit;
    const int64_t s0 = (int64_t)blockIdx.y * per;
    const int KT = (int)(steps - s0 < per ? (steps - s0 > 0 ? steps - s0 : 0) : per);

    auto issue = [&](int kt) {
        char* st = smem + (kt % NS) * STAGE;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            su.issue(st + k * SideU::BYTES, k * p.u.stride * 2, s0 + kt, kt < KT, wave, lane);
            sv.issue(st + NP * SideU::BYTES + k * SideV::BYTES, k * p.v.stride * 2, s0 + kt, kt < KT, wave, lane);
        }
    };
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // fragments are read one step ahead, into the other of two register sets
    struct Frags {
        i32x4 a[FI][NP], b[FJ][NP];
    };
    auto read = [&](Frags& f, int kt) {
        const char* st = smem + (kt % NS) * STAGE;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
#pragma unroll
            for (int j = 0; j < FJ; ++j) f.b[j][k] = SideV::frag(st + NP * SideU::BYTES + k * SideV::BYTES, wj * WJ + j * 16, lane);
#pragma unroll
            for (int i = 0; i < FI; ++i) f.a[i][k] = SideU::frag(st + k * SideU::BYTES, wi * WI + i * 16, lane);
        }
    };
    // step kt's MFMAs, from `f`; step kt+1's fragments into `nx`.  Before them:
    // the wave holds all of stage kt, step kt+1 has landed, and stage kt is
    // free for step kt+NS.  (Steps past the last read zeros.)
    auto step = [&](int kt, const Frags& f, Frags& nx) {
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        wait_vm<(NS - 2) * Q>();
        lds_barrier();
        issue(kt + NS);
        __builtin_amdgcn_sched_barrier(0);
        read(nx, kt + 1);
        piece_mma<NP>(f.a, f.b, acc);
        if constexpr (!TRU && !TRV) {
            // a fragment read, then its share of the MFMAs (left alone, the
            // compiler sinks the reads below them; with transposing reads, two
            // halves a fragment, it took 112 us for 107 and registers spilled)
            constexpr int ND = NP * (FI + FJ), NM = FI * FJ * NP * (NP + 1) / 2;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, NM / ND, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, NM - NM / ND * ND, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    if (KT > 0) {
        Frags f0, f1;
#pragma unroll
        for (int s = 0; s < NS; ++s) issue(s);
        wait_vm<(NS - 1) * Q>();
        lds_barrier();
        read(f0, 0);
        for (int kt = 0; kt < KT; kt += 2) {
            step(kt, f0, f1);
            step(kt + 1, f1, f0);
        }
    }
    wait_vm<0>();
    const int g = lane >> 4, r = lane & 15;
#pragma unroll
    for (int i = 0; i < FI; ++i) {
        const int64_t oi = i0 + wi * WI + i * 16 + 4 * g;
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
            const int64_t oj = j0 + wj * WJ + j * 16 + r;
            if (oj >= p.J) continue;
            if (p.ksplit > 1 || p.sym) {
                const int64_t ldp = (p.I + 3) & ~(int64_t)3;
                if (oi < ldp) *(f32x4*)(p.partial + ((int64_t)blockIdx.y * p.J + oj) * ldp + oi) = acc[i][j];
            } else {
                ns_finish4<NP>(p, exps, acc[i][j], oj, oi);
            }
        }
    }
}

// sums of the K splits in split order, then the same finish
template <int NP>
__global__ __launch_bounds__(256) void ns_reduce_kernel(NsParams p) {
    const NsExps exps(p);
    const int64_t ldp = (p.I + 3) & ~(int64_t)3;
    // (pieces: up to the padded row end, whose last four are zeros)
    const int64_t q = (p.mode == NS_OUT ? ldp : p.o.ld) / 4;
    const int64_t total = p.J * q;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t j = t / q, i = (t - j * q) * 4;
        f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
        if (i < ldp)
            for (int k = 0; k < p.ksplit; ++k) s += *(const f32x4*)(p.partial + ((int64_t)k * p.J + j) * ldp + i);
        ns_finish4<NP>(p, exps, s, j, i);
    }
}

// The same for a symmetric output of which the tiles reaching i >= j were
// computed: a 64 x 64 block with i >= j a workgroup (tiles are multiples of
// 64, so every such block is whole), written as it is and mirrored through LDS.
template <int NP>
__global__ __launch_bounds__(256) void ns_sym_reduce_kernel(NsParams p) {
    const NsExps exps(p);
    __shared__ float tile[64][65];
    const int64_t ldp = (p.I + 3) & ~(int64_t)3;
    int bi = 0, bj = blockIdx.x;
    while (bj > bi) bj -= ++bi;
    const int row = threadIdx.x >> 4, quad = (threadIdx.x & 15) * 4;
    const int64_t i = (int64_t)bi * 64 + quad;
    f32x4 s[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 3
    for (int k = 0; k < p.ksplit; ++k) {
        f32x4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t j = (int64_t)bj * 64 + u * 16 + row;
            w[u] = j < p.J && i < ldp ? *(const f32x4*)(p.partial + ((int64_t)k * p.J + j) * ldp + i) : f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] += w[u];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t j = (int64_t)bj * 64 + u * 16 + row;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (j < p.J && i < p.o.ld) {
            ns_values4<NP>(p, exps, s[u], j, i, v);
            ns_store4<NP>(p, v, j, i);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) tile[u * 16 + row][quad + e] = v[e];
    }
    if (bi == bj) return;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t j = (int64_t)bi * 64 + u * 16 + row;
        if (j >= p.J) continue;   // (the columns are inside: block bj is before the last)
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = tile[quad + e][u * 16 + row];
        ns_store4<NP>(p, v, j, (int64_t)bj * 64 + quad);
    }
}

// ---- thin updates (a LoRA factor's): the iteration on the n x n side -----------------
//
// For n <= 128 one step's work is small and its launches and passes over X
// are not.  Every matrix of the iteration is a polynomial of the first A, so
// they commute, and several steps need X only at their ends:
//   P = a I + b A + c A^2,   Q <- P Q,   A <- P A P,     then X <- Q X.
// One workgroup runs a segment of steps on A in LDS; one pass over X applies
// Q, and takes the next segment's Gram matrix while X is there.  A's rounding
// errors grow by a^2 a step against its small eigenvalues (twice as fast as
// X's own), so a segment has at most 3 steps with two pieces (its errors stay
// near 1e-5 of the result, a hundredth of a 16-bit rounding; all 5 steps in
// one segment measured 1e-4 and more), and one step with three.
// Times at bf16 8192 x 128 / bf16 16 x 4096 / fp32 64 x 4096, us a launch:
//   ns_chunk_kernel  Gram matrix of X / X <- Q X with it / the last X <- Q X:
//                    10.5, 14.8, 8.3 / 4.1, -, 5.4 / 5.3, 7.4, 6.1 (launch, one round of
//                    loads, LDS and the Gram matrices' writes; no bandwidth near its limit)
//   Iter             a segment of steps; the first one scales by 1 / (|G| + eps),
//                    |G|^2 being the trace: 29 and 19 (9 and 5 dependent 128^3
//                    products) / 7.3 (in 64 bits) / 3.9
//                    (a kernel of its own: run by the last workgroup of the one
//                    before, behind a device-wide fence, it took 2 us more)
//   ns_sum_kernel    the workgroups' Gram matrices added up (n > 32): 4.5 / - / 3.3

constexpr int NS_SEG = 3, NS_SEG64 = 5;
constexpr double NS_QMAX = 1024.0;   // bound on Q's largest factor within a segment
constexpr int NS_THIN = 128;
constexpr int NS_EMPTY = -100000;   // exponent of a workgroup that saw zeros only

template <int NPAD>
struct ThinShape {
    static constexpr int NW = NPAD == 128 ? 8 : 4, NT = NW * 64;
    static constexpr int CW = NPAD == 16 ? 256 : NPAD == 32 ? 128 : 64;   // columns a chunk
    static constexpr int LD = CW + 8;            // LDS row: consecutive rows four banks on
    static constexpr int KR = NPAD < 32 ? 32 : NPAD;   // rows an MFMA step reads (zeros past NPAD)
    static constexpr int IB = NPAD / 16, WC = NW / IB, CB = CW / 16 / WC;
    static constexpr int PT = NPAD * CW / NT;    // elements a thread loads
    static constexpr int GT = NPAD == 16 ? 1 : IB * IB / NW;   // Gram tiles a wave
    static constexpr bool KSPLIT = NPAD == 16;   // one Gram tile: the waves share its columns
    static_assert(CB == 4 && PT == 16, "a chunk's shares");
};

struct ThinParams {
    const void* g;      // raw source [R][C] (src 0: wide, 1: tall)
    int src, dt;        // 2: x, fp32 [n][ldx]
    int vec;            // 8-element runs of the source are whole and 16-byte aligned
    int64_t n, m, ldx;
    float* x;
    const uint16_t* q;  // pieces [NP][NPAD][KR], scaled
    const double* fac;  // X' = fac * 2^e * (q . pieces)
    float* part;        // a Gram matrix per workgroup, [NPAD][NPAD]
    int* exps;          // which stands for 2^(2 e) times its values
    int* chunk_e;       // x's chunks' exponents (two pieces)
    void* out;          // [R][C]
    int tall;
    int vec_out;        // out's rows hold whole groups of 4 elements, aligned for one store each
};

// the largest of a wave's values, in every lane
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    auto step = [&](uint32_t o) { v = o > v ? o : v; };
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));   // row_shr 1, 2, 4, 8
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xF, 0xF, false));   // row_bcast 15, 31
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xF, 0xF, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ int exponent_of(uint32_t abs_bits) { return (int)(abs_bits >> 23) - 127; }

// 8 consecutive rows of one column of an LDS tile [row][LD]: the transposing
// read of lyc_device.h's frag_t, rows LD elements apart
template <int LD>
__device__ __forceinline__ i32x4 thin_frag_t(const uint16_t* t, int row0, int col0, int lane) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const int G = lane >> 4, j = lane & 15;
    const uint16_t* p = t + (row0 + 8 * G + (j >> 2)) * LD + col0 + 4 * (j & 3);
    const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(__attribute__((address_space(3))) uint16_t*)p);
    const s4 b =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(__attribute__((address_space(3))) uint16_t*)(p + 4 * LD));
    const i32x2 ai = __builtin_bit_cast(i32x2, a), bi = __builtin_bit_cast(i32x2, b);
    return i32x4{ai[0], ai[1], bi[0], bi[1]};
}

struct IterParams {
    const float* part;   // Gram matrices [slots][NPAD][NPAD], standing for 2^(2 e) times their values
    const int* exps;     // e of each
    int slots, steps, first;
    float a, b, c;
    double eps;
    float sA[NS_SEG], sP[NS_SEG], sT[NS_SEG], sQ[NS_SEG];   // the powers of two fp16 pieces are held times, step by step
    uint16_t* q;         // pieces [NP][NPAD][KR]
    double* fac;
};

// the largest of the slots' exponents
__device__ __forceinline__ int top_exponent(const int* exps, int slots) {
    int e = NS_EMPTY;
    for (int i = threadIdx.x & 63; i < slots; i += 64) e = exps[i] > e ? exps[i] : e;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_xor(e, d);
        e = o > e ? o : e;
    }
    return e;
}
__device__ __forceinline__ float slot_weight(int e, int top) {
    const int d = 2 * (e - top);
    return d < -126 ? 0.f : __builtin_ldexpf(1.f, d);
}

// A segment on the n x n side, by one workgroup: waves WB (WB + 1) / 2 hold the
// blocks on and below the diagonal (every matrix is symmetric), masters in
// registers in MFMA layout; operands go to LDS whole, as pieces, a block and
// its mirror image, and serve as either operand row by row.
constexpr int iter_threads(int npad) { return npad == 16 ? 64 : npad == 32 ? 192 : 640; }

template <int NPAD, int NP>
struct Iter {
    static constexpr int IB = NPAD / 16;
    static constexpr int TW = NPAD == 128 ? 2 : 1;   // tiles per wave along each side
    static constexpr int WB = IB / TW, WAVES = WB * (WB + 1) / 2;
    static_assert(WAVES * 64 == iter_threads(NPAD), "launch");
    static constexpr int KR = NPAD < 32 ? 32 : NPAD, LD = KR + 8, KS = KR / 32;
    static constexpr int BUFS = NP == 2 ? 2 : 1;
    static constexpr int LDS = BUFS * NP * NPAD * LD * 2;   // bytes
    typedef f32x4 M[TW][TW];

    uint16_t* buf;   // [BUFS][NP][NPAD * LD]
    int lane, g, r, wi, wj;

    __device__ __forceinline__ int row_of(int ti) const { return (wi * TW + ti) * 16 + 4 * g; }   // first of 4 rows
    __device__ __forceinline__ int col_of(int tj) const { return (wj * TW + tj) * 16 + r; }
    __device__ __forceinline__ uint16_t* at(int b, int k) const { return buf + (b * NP + k) * NPAD * LD; }

    // 2^ex v (bf16 pieces have fp32's range and are taken as they are)
    static __device__ __forceinline__ float held(float v, float scale) { return NP == 2 ? v * scale : v; }

    __device__ __forceinline__ void put(int b, const M& m, float scale) const {
#pragma unroll
        for (int ti = 0; ti < TW; ++ti)
#pragma unroll
            for (int tj = 0; tj < TW; ++tj) {
                uint16_t o[4][NP];
#pragma unroll
                for (int e = 0; e < 4; ++e) Pieces<NP>::split(held(m[ti][tj][e], scale), o[e]);
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    *(i32x2*)(at(b, k) + col_of(tj) * LD + row_of(ti)) =
                        i32x2{(int)((uint32_t)o[0][k] | (uint32_t)o[1][k] << 16),
                              (int)((uint32_t)o[2][k] | (uint32_t)o[3][k] << 16)};
                    if (wi != wj) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) at(b, k)[(row_of(ti) + e) * LD + col_of(tj)] = o[e][k];
                    }
                }
            }
    }
    __device__ __forceinline__ void product(int bu, int bv, float scale, M& out) const {
#pragma unroll
        for (int ti = 0; ti < TW; ++ti)
#pragma unroll
            for (int tj = 0; tj < TW; ++tj) out[ti][tj] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            i32x4 u[TW][NP], v[TW][NP];
#pragma unroll
            for (int t = 0; t < TW; ++t)
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    u[t][k] = *(const i32x4*)(at(bu, k) + ((wi * TW + t) * 16 + r) * LD + s * 32 + g * 8);
                    v[t][k] = *(const i32x4*)(at(bv, k) + ((wj * TW + t) * 16 + r) * LD + s * 32 + g * 8);
                }
            piece_mma<NP>(u, v, out);
        }
        if constexpr (NP == 2) {
#pragma unroll
            for (int ti = 0; ti < TW; ++ti)
#pragma unroll
                for (int tj = 0; tj < TW; ++tj) out[ti][tj] *= scale;
        }
    }

    // all of the workgroup's WAVES * 64 threads
    __device__ void run(const IterParams& p, char* lds, float* diag) {
        constexpr int nt = WAVES * 64;
        const int tid = threadIdx.x;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        lane = tid & 63;
        g = lane >> 4;
        r = lane & 15;
        buf = (uint16_t*)lds;
        wi = 0;
        while ((wi + 1) * (wi + 2) / 2 <= wave) ++wi;
        wj = wave - wi * (wi + 1) / 2;
        // zero the columns an MFMA step reads past NPAD
        if constexpr (KR > NPAD) {
            for (int i = tid; i < BUFS * NP * NPAD * LD; i += nt) buf[i] = 0;
            __syncthreads();
        }
        const int top = top_exponent(p.exps, p.slots);
        M A, Q;
#pragma unroll
        for (int ti = 0; ti < TW; ++ti)
#pragma unroll
            for (int tj = 0; tj < TW; ++tj) {
                const int64_t o = (int64_t)col_of(tj) * NPAD + row_of(ti);
                f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 16
                for (int k = 0; k < p.slots; ++k)
                    s += *(const f32x4*)(p.part + (int64_t)k * NPAD * NPAD + o) * slot_weight(p.exps[k], top);
                A[ti][tj] = s;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (row_of(ti) + e == col_of(tj)) diag[col_of(tj)] = s[e];
            }
        // A's true size is 2^(2 top) times its values; the first segment divides by (|G| + eps)^2
        double inv = 1.0;
        if (p.first) {
            __syncthreads();
            double tr = 0;
            for (int i = lane; i < NPAD; i += 64) tr += (double)diag[i];
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) tr += __shfl_xor(tr, d);
            const double norm = top == NS_EMPTY ? 0.0 : __builtin_ldexp(__builtin_sqrt(tr), top);
            inv = ns_inverse(norm, p.eps);
        }
        const double half = top == NS_EMPTY ? 0.0 : __builtin_ldexp(inv, top);
        const float fA = (float)(half * half);
#pragma unroll
        for (int ti = 0; ti < TW; ++ti)
#pragma unroll
            for (int tj = 0; tj < TW; ++tj) A[ti][tj] *= fA;

        for (int k = 0; k < p.steps; ++k) {
            M P;
            put(0, A, p.sA[k]);
            __syncthreads();
            product(0, 0, 1.f / (p.sA[k] * p.sA[k]), P);
#pragma unroll
            for (int ti = 0; ti < TW; ++ti)
#pragma unroll
                for (int tj = 0; tj < TW; ++tj)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // (A^2 may leave fp32's range where nothing takes it)
                        float v = (p.c != 0.f ? p.c * P[ti][tj][e] : 0.f) + p.b * A[ti][tj][e];
                        if (row_of(ti) + e == col_of(tj)) v += p.a;
                        P[ti][tj][e] = v;
                    }
            const bool more = k + 1 < p.steps;
            if constexpr (NP == 2) {
                if (k > 0 || more) {
                    put(1, P, p.sP[k]);
                    __syncthreads();
                }
                if (more) product(0, 1, 1.f / (p.sA[k] * p.sP[k]), A);   // T = A P
                if (k > 0) {
                    __syncthreads();   // buffer 0 has been read
                    put(0, Q, p.sQ[k - 1]);
                    __syncthreads();
                    product(0, 1, 1.f / (p.sQ[k - 1] * p.sP[k]), Q);
                }
                if (more) {
                    __syncthreads();
                    put(0, A, p.sT[k]);
                    __syncthreads();
                    product(0, 1, 1.f / (p.sT[k] * p.sP[k]), A);   // P A P
                    __syncthreads();
                }
            }
            if (k == 0) {
#pragma unroll
                for (int ti = 0; ti < TW; ++ti)
#pragma unroll
                    for (int tj = 0; tj < TW; ++tj) Q[ti][tj] = P[ti][tj];
            }
        }
        const float sq = NP == 2 ? p.sQ[p.steps - 1] : 1.f;
#pragma unroll
        for (int ti = 0; ti < TW; ++ti)
#pragma unroll
            for (int tj = 0; tj < TW; ++tj) {
                uint16_t o[4][NP];
#pragma unroll
                for (int e = 0; e < 4; ++e) Pieces<NP>::split(held(Q[ti][tj][e], sq), o[e]);
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    uint16_t* q = p.q + (int64_t)k * NPAD * KR;
                    *(i32x2*)(q + col_of(tj) * KR + row_of(ti)) =
                        i32x2{(int)((uint32_t)o[0][k] | (uint32_t)o[1][k] << 16),
                              (int)((uint32_t)o[2][k] | (uint32_t)o[3][k] << 16)};
                    if (wi != wj) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) q[(row_of(ti) + e) * KR + col_of(tj)] = o[e][k];
                    }
                }
            }
        if constexpr (KR > NPAD) {
            for (int i = tid; i < NP * NPAD * (KR - NPAD); i += nt)
                p.q[(i / (KR - NPAD)) * KR + NPAD + i % (KR - NPAD)] = 0;
        }
        if (tid == 0) *p.fac = inv / (double)sq;
    }
};

// sum = the Gram matrices added up at the largest exponent, four floats a
// thread; 8 threads share an element's slots, added in thread order
__global__ __launch_bounds__(256) void ns_sum_kernel(const float* part, const int* exps, int slots, int quads, float* sum,
                                                     int* top_out) {
    __shared__ __attribute__((aligned(16))) f32x4 red[8][32];
    const int tid = threadIdx.x, e = tid & 31, h = tid >> 5;
    const int top = top_exponent(exps, slots);
    const int at = (int)blockIdx.x * 32 + e;
    f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
    if (at < quads) {
#pragma unroll 8
        for (int k = h; k < slots; k += 8) s += *(const f32x4*)(part + ((int64_t)k * quads + at) * 4) * slot_weight(exps[k], top);
    }
    red[h][e] = s;
    __syncthreads();
    if (h == 0 && at < quads) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += red[k][e];
        *(f32x4*)(sum + (int64_t)at * 4) = s;
        if (blockIdx.x == 0 && tid == 0) *top_out = top;
    }
}

// The segment for n <= 16 and a 16-bit G, by one wave in 64 bits, all of it in
// registers: v_mfma_f64_16x16x4 leaves lane (r = lane % 16, g = lane / 16) the
// elements (4 e + g, r), and takes as step s of either operand the element
// (r, 4 s + g), which for a symmetric matrix is the same register.  A product
// is four MFMAs and nothing else, and 64 bits leave no growth of errors to
// stop for: five steps a segment (17 products, about 3 us).
typedef double f64x4 __attribute__((ext_vector_type(4)));
__global__ __launch_bounds__(64) void ns_iter64_kernel(IterParams p) {
    constexpr int KR = ThinShape<16>::KR;
    const int lane = threadIdx.x, g = lane >> 4, r = lane & 15;
    const int top = top_exponent(p.exps, p.slots);
    f64x4 A = f64x4{0, 0, 0, 0};
#pragma unroll 8
    for (int k = 0; k < p.slots; ++k) {
        const double w = (double)slot_weight(p.exps[k], top);
#pragma unroll
        for (int e = 0; e < 4; ++e) A[e] += w * (double)p.part[k * 256 + r * 16 + 4 * e + g];
    }
    double inv = 1.0;
    if (p.first) {
        double tr = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) tr += 4 * e + g == r ? A[e] : 0.0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) tr += __shfl_xor(tr, d);
        inv = ns_inverse(top == NS_EMPTY ? 0.0 : __builtin_ldexp(__builtin_sqrt(tr), top), p.eps);
    }
    const double half = top == NS_EMPTY ? 0.0 : __builtin_ldexp(inv, top);
    A *= half * half;
    auto product = [](const f64x4& u, const f64x4& v) {
        f64x4 c = f64x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f64_16x16x4f64(u[s], v[s], c, 0, 0, 0);
        return c;
    };
    f64x4 Q = f64x4{0, 0, 0, 0};
    for (int k = 0; k < p.steps; ++k) {
        f64x4 P = product(A, A);
#pragma unroll
        for (int e = 0; e < 4; ++e) P[e] = (double)p.c * P[e] + (double)p.b * A[e] + (4 * e + g == r ? (double)p.a : 0.0);
        Q = k == 0 ? P : product(Q, P);
        if (k + 1 < p.steps) A = product(product(A, P), P);
    }
    const float sq = p.sQ[0];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint16_t o[2];
        Pieces<2>::split((float)(Q[e] * (double)sq), o);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            p.q[(k * 16 + r) * KR + 4 * e + g] = o[k];
            p.q[(k * 16 + r) * KR + 16 + 4 * e + g] = 0;
        }
    }
    if (lane == 0) *p.fac = inv / (double)sq;
}

template <int NPAD, int NP>
__global__ __launch_bounds__(iter_threads(NPAD)) void ns_iter_kernel(IterParams p) {
    using I = Iter<NPAD, NP>;
    __shared__ __attribute__((aligned(16))) char lds[I::LDS];
    __shared__ float diag[NPAD];
    I it;
    it.run(p, lds, diag);
}

enum { THIN_GRAM = 0, THIN_BOTH = 1, THIN_OUT = 2 };

template <int NPAD, int NP, int MODE>
__global__ __launch_bounds__(ThinShape<NPAD>::NT) void ns_chunk_kernel(ThinParams p) {
    using S = ThinShape<NPAD>;
    constexpr int LD = S::LD, CW = S::CW, KS = S::KR / 32;
    __shared__ __attribute__((aligned(16))) uint16_t xs[NP][S::KR * LD];
    __shared__ uint32_t wmax[S::NW];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ib = wave % S::IB, cb0 = wave / S::IB * S::CB;
    if constexpr (S::KR > NPAD) {
        for (int i = tid; i < (S::KR - NPAD) * LD; i += S::NT)
#pragma unroll
            for (int k = 0; k < NP; ++k) xs[k][NPAD * LD + i] = 0;
    }
    i32x4 q[KS][1][NP];
    float fac = 0;   // X' = 2^(fexp + e) fac (q . pieces)
    int fexp = 0;
    if constexpr (MODE != THIN_GRAM) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int k = 0; k < NP; ++k)
                q[s][0][k] = *(const i32x4*)(p.q + ((int64_t)k * NPAD + ib * 16 + r) * S::KR + s * 32 + g * 8);
        fac = (float)frexp(*p.fac, &fexp);
    }
    f32x4 gacc[1][S::GT];
#pragma unroll
    for (int t = 0; t < S::GT; ++t) gacc[0][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Pieces of X are taken from a chunk scaled by 2^-e, its largest magnitude
    // to [2^11, 2^12) (fp16 pieces' low bits stay normal; subnormal maxima count
    // as 2^-126).  The chunks of a Gram matrix share the largest e so far, the
    // sums made with a smaller one are scaled down.
    int erun = NS_EMPTY;
    auto group_max = [&]() {
        uint32_t v = wmax[0];
#pragma unroll
        for (int w = 1; w < S::NW; ++w) v = wmax[w] > v ? wmax[w] : v;
        return v;
    };
    auto chunk_exponent = [](uint32_t top) { return exponent_of(top < 0x00800000u ? 0x00800000u : top) - 11; };
    auto gram_exponent = [&](int e) {
        if (erun == NS_EMPTY) erun = e;
        else if (e > erun) {
            const float f = __builtin_ldexpf(1.f, 2 * (erun - e) < -126 ? -126 : 2 * (erun - e));
#pragma unroll
            for (int t = 0; t < S::GT; ++t) gacc[0][t] *= f;
            erun = e;
        }
        return erun;
    };

    const int64_t chunks = (p.m + CW - 1) / CW;
    for (int64_t ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
        const int64_t c0 = ch * CW;
        int x_exponent = 0;
        if constexpr (NP == 2 && MODE != THIN_GRAM) {
            if (p.src == 2) x_exponent = p.chunk_e[ch];
        }
        // the chunk, 16 elements a thread: two runs of 8 along the stored rows
        // where those are whole 16-byte pieces (vec), else single elements
        float v[S::PT];
        int row0[2], col0[2];   // of the runs
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t8 = tid + h * S::NT;
            // (tall: 16 consecutive stored rows a group of lanes, so that the
            // transposed LDS writes fall on few common banks)
            row0[h] = p.src == 1 ? (t8 >> 4) % (NPAD / 8) * 8 : t8 / (CW / 8);
            col0[h] = p.src == 1 ? t8 / (2 * NPAD) * 16 + (t8 & 15) : t8 % (CW / 8) * 8;
        }
        const bool f32 = p.src == 2 || p.dt == DT_F32;
        const auto rs = make_rsrc(p.src == 2 ? (const void*)p.x : p.g,
                                  (uint32_t)(p.src == 2 ? p.n * p.ldx * 4 : p.n * p.m * (f32 ? 4 : 2)));
        const uint32_t ld = (uint32_t)(p.src == 1 ? p.n : p.src == 2 ? p.ldx : p.m);
        // byte offset of an element, out of range where there is none
        auto offset = [&](int row, int col) -> uint32_t {
            if (row >= p.n || c0 + col >= p.m) return OOB;
            return (p.src == 1 ? (uint32_t)(c0 + col) * ld + (uint32_t)row : (uint32_t)row * ld + (uint32_t)(c0 + col)) *
                   (f32 ? 4u : 2u);
        };
        auto widen = [&](uint32_t b) { return p.dt == DT_F16 ? f16_to_f32((uint16_t)b) : bf16_to_f32((uint16_t)b); };
        if (p.vec) {
            i32x4 raw[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t o = offset(row0[h], col0[h]);
                raw[h][0] = buf_load16(rs, o);
                raw[h][1] = buf_load16(rs, f32 ? o + 16 : OOB);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint32_t w = (uint32_t)raw[h][0][u >> 1];
                    const float half = widen((u & 1) ? w >> 16 : w);
                    v[8 * h + u] = f32 ? __builtin_bit_cast(float, (uint32_t)raw[h][u >> 2][u & 3]) : half;
                }
        } else {
            uint32_t raw[S::PT];
#pragma unroll
            for (int u = 0; u < S::PT; ++u) {
                const uint32_t o = offset(row0[u >> 3] + (p.src == 1 ? u & 7 : 0), col0[u >> 3] + (p.src == 1 ? 0 : u & 7));
                raw[u] = f32 ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, o, 0, 0)
                             : (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, o, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < S::PT; ++u) v[u] = f32 ? __builtin_bit_cast(float, raw[u]) : widen(raw[u]);
        }
        // (X between the segments: the pass that stored it knows; bf16 pieces have
        // fp32's range and take it as it is)
        int e = 0;
        if (p.src != 2) {
            uint32_t mx = 0;
#pragma unroll
            for (int u = 0; u < S::PT; ++u) {
                const uint32_t b = __builtin_bit_cast(uint32_t, v[u]) & 0x7FFFFFFFu;
                mx = b > mx ? b : mx;
            }
            mx = wave_max(mx);
            if (lane == 0) wmax[wave] = mx;
            __syncthreads();   // (the previous chunk's tile has been read, too)
            mx = group_max();
            if (mx != 0) e = chunk_exponent(mx);
            if constexpr (MODE == THIN_GRAM) {
                if (mx == 0) {
                    __syncthreads();   // (wmax is read by all before the next chunk writes it)
                    continue;          // zeros add nothing
                }
                e = gram_exponent(e);
            }
        } else {
            if constexpr (NP == 2 && MODE != THIN_GRAM) e = x_exponent;
            __syncthreads();   // the previous chunk's tile has been read
        }
        const Pow2 scaled(-e);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint16_t o[8][NP];
#pragma unroll
            for (int u = 0; u < 8; ++u) Pieces<NP>::split(scaled(v[8 * h + u]), o[u]);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                if (p.src == 1) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) xs[k][(row0[h] + u) * LD + col0[h]] = o[u][k];
                } else {
                    i32x4 w;
#pragma unroll
                    for (int u = 0; u < 4; ++u) w[u] = (int)((uint32_t)o[2 * u][k] | (uint32_t)o[2 * u + 1][k] << 16);
                    *(i32x4*)&xs[k][row0[h] * LD + col0[h]] = w;
                }
            }
        }
        __syncthreads();

        if constexpr (MODE != THIN_GRAM) {
            // (a factor and an exponent: the two together may leave fp32's range)
            const Pow2 fe(fexp + e);
            const float fa = fac * fe.a;
            auto finished = [&](float s) { return s * fa * fe.b; };
            f32x4 acc[S::CB][1];
#pragma unroll
            for (int c = 0; c < S::CB; ++c) acc[c][0] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s)
            {
                i32x4 x[S::CB][NP];
#pragma unroll
                for (int c = 0; c < S::CB; ++c)
#pragma unroll
                    for (int k = 0; k < NP; ++k) x[c][k] = thin_frag_t<LD>(xs[k], s * 32, (cb0 + c) * 16, lane);
                // (tall: the transposed tile, 4 consecutive i a lane)
                if (MODE == THIN_OUT && p.tall) piece_mma<NP>(q[s], x, *(f32x4(*)[1][S::CB])&acc);
                else piece_mma<NP>(x, q[s], acc);
            }
            if constexpr (MODE == THIN_OUT) {
#pragma unroll
                for (int c = 0; c < S::CB; ++c) {
                    // wide: row i of the block, 4 consecutive columns; tall: the other way round
                    const int64_t i = ib * 16 + (p.tall ? 4 * g : r), cc = c0 + (cb0 + c) * 16 + (p.tall ? r : 4 * g);
                    if (p.vec_out) {   // the four are inside the row, or none is
                        if (i >= p.n || cc >= p.m) continue;
                        f32x4 val;
#pragma unroll
                        for (int el = 0; el < 4; ++el) val[el] = finished(acc[c][0][el]);
                        const int64_t o = p.tall ? cc * p.n + i : i * p.m + cc;
                        if (p.dt == DT_F32) {
                            *(f32x4*)((float*)p.out + o) = val;
                        } else {
                            const bool h = p.dt == DT_F16;
                            const uint32_t lo = h ? pack_f16x2(val[0], val[1]) : pack_bf16x2(val[0], val[1]);
                            const uint32_t hi = h ? pack_f16x2(val[2], val[3]) : pack_bf16x2(val[2], val[3]);
                            *(i32x2*)((uint16_t*)p.out + o) = i32x2{(int)lo, (int)hi};
                        }
                        continue;
                    }
#pragma unroll
                    for (int el = 0; el < 4; ++el) {
                        const int64_t ie = p.tall ? i + el : i, ce = p.tall ? cc : cc + el;
                        if (ie >= p.n || ce >= p.m) continue;
                        const int64_t o = p.tall ? ce * p.n + ie : ie * p.m + ce;
                        const float val = finished(acc[c][0][el]);
                        if (p.dt == DT_F32) ((float*)p.out)[o] = val;
                        else ((uint16_t*)p.out)[o] = p.dt == DT_F16 ? f32_to_f16(val) : f32_to_bf16(val);
                    }
                }
                continue;
            } else {
                const int i = ib * 16 + r;
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < S::CB; ++c) {
#pragma unroll
                    for (int el = 0; el < 4; ++el) {
                        acc[c][0][el] = finished(acc[c][0][el]);
                        const float val = acc[c][0][el];
                        const uint32_t b = __builtin_bit_cast(uint32_t, val) & 0x7FFFFFFFu;
                        top = b > top ? b : top;
                    }
                    if (i < p.n) *(f32x4*)(p.x + i * p.ldx + c0 + (cb0 + c) * 16 + 4 * g) = acc[c][0];
                }
                int en = 0;
                if constexpr (NP == 2) {
                    top = wave_max(top);
                    if (lane == 0) wmax[wave] = top;
                    __syncthreads();   // the tile has been read: X' takes its place
                    top = group_max();
                    en = top == 0 ? 0 : chunk_exponent(top);
                    if (tid == 0) p.chunk_e[ch] = en;
                    if (top == 0) {
                        __syncthreads();
                        continue;
                    }
                    en = gram_exponent(en);
                } else {
                    __syncthreads();   // the tile has been read: X' takes its place
                    erun = 0;
                }
                const Pow2 scaled_next(-en);
#pragma unroll
                for (int c = 0; c < S::CB; ++c) {
                    const int cc = (cb0 + c) * 16 + 4 * g;
                    uint16_t o[4][NP];
#pragma unroll
                    for (int el = 0; el < 4; ++el) Pieces<NP>::split(scaled_next(acc[c][0][el]), o[el]);
#pragma unroll
                    for (int k = 0; k < NP; ++k)
                        *(i32x2*)&xs[k][i * LD + cc] = i32x2{(int)((uint32_t)o[0][k] | (uint32_t)o[1][k] << 16),
                                                             (int)((uint32_t)o[2][k] | (uint32_t)o[3][k] << 16)};
                }
                __syncthreads();
            }
        }
        if constexpr (MODE != THIN_OUT) {
            constexpr int GK = CW / 32 / (S::KSPLIT ? S::NW : 1);
#pragma unroll
            for (int s = 0; s < GK; ++s) {
                const int ks = S::KSPLIT ? wave * GK + s : s;
                const int gi = S::KSPLIT ? 0 : wave % S::IB;
                i32x4 a[1][NP], b[S::GT][NP];
#pragma unroll
                for (int k = 0; k < NP; ++k) a[0][k] = *(const i32x4*)&xs[k][(gi * 16 + r) * LD + ks * 32 + g * 8];
#pragma unroll
                for (int t = 0; t < S::GT; ++t) {
                    const int gj = S::KSPLIT ? 0 : wave / S::IB * S::GT + t;
#pragma unroll
                    for (int k = 0; k < NP; ++k) b[t][k] = *(const i32x4*)&xs[k][(gj * 16 + r) * LD + ks * 32 + g * 8];
                }
                piece_mma<NP>(a, b, gacc);
            }
        }
    }
    if constexpr (MODE != THIN_OUT) {
        if constexpr (S::KSPLIT) {
            __syncthreads();   // the last chunk's tile has been read
            f32x4* red = (f32x4*)&xs[0][0];
            red[wave * 64 + lane] = gacc[0][0];
            __syncthreads();
            gacc[0][0] = red[lane];
#pragma unroll
            for (int w = 1; w < S::NW; ++w) gacc[0][0] += red[w * 64 + lane];
        }
        const int gi = S::KSPLIT ? 0 : wave % S::IB;
#pragma unroll
        for (int t = 0; t < S::GT; ++t) {
            const int gj = S::KSPLIT ? 0 : wave / S::IB * S::GT + t;
            if (!S::KSPLIT || wave == 0)
                *(f32x4*)(p.part + ((int64_t)blockIdx.x * NPAD + gj * 16 + r) * NPAD + gi * 16 + 4 * g) = gacc[0][t];
        }
        if (tid == 0) p.exps[blockIdx.x] = erun;
    }
}

// ---- host ----------------------------------------------------------------------------------

static int64_t up8(int64_t v) { return (v + 7) & ~(int64_t)7; }
static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Tile and K split of an I x J product over K, by modelled time: rounds of
// workgroups over the CUs (two of the small tile's share one) times a fixed
// part and a K step's as measured, plus the partial sums' round trip of a
// split.  A symmetric output (A and P) may take the tiles that reach i >= j
// alone, about half, with more splits to fill the device, and a reduction that
// mirrors them.  us:
//   A of 2048 x 4096, two pieces: 100 in 128 x 128 tiles, 107 in 256 x 128
//     tiles with two splits; halved, 256 x 128, three splits: 64 + 11
//   A^2 there: 67 in 128 x 128 tiles; halved as above: 37 + 11
//   4096 x 2048 over 2048, X transposed: 119 in 128 x 128, 107 in 256 x 128
//   400 x 400 over 600, three pieces, four splits: 13.4 in 128 x 128 tiles, 8.2
//     in 64 x 64
// (Three pieces: the large tile's fragments do not fit the registers.)
enum { NS_256x128, NS_128x128, NS_64x64 };
struct NsPlan {
    int tile, ksplit, sym, blocks;   // blocks: workgroups of one split
};
static NsPlan ns_plan(int64_t I, int64_t J, int64_t K, int np, bool symmetric) {
    struct C { int id, ti, tj, per_cu; double fixed, step2, step3; };   // us
    const C cands[] = {{NS_256x128, 256, 128, 1, 9.0, 1.30, 0.0}, {NS_128x128, 128, 128, 1, 6.5, 0.76, 1.25},
                       {NS_64x64, 64, 64, 2, 3.3, 0.70, 1.0}};
    const double cus = (double)device_rates().cus;
    const int64_t steps = (K + 31) / 32;
    double best = 1e300;
    NsPlan plan{NS_64x64, 1, 0, 0};
    for (const C& c : cands) {
        if (c.id == NS_256x128 && np != 2) continue;
        const int64_t ni = (I + c.ti - 1) / c.ti, nj = (J + c.tj - 1) / c.tj;
        for (int sym = 0; sym <= (symmetric ? 1 : 0); ++sym) {
            int64_t blocks = sym ? 0 : ni * nj;
            if (sym)
                for (int64_t i = 0; i < ni; ++i) blocks += sym_tiles((int)i, c.ti, c.tj, (int)nj);
            for (int u = 0; u < 12; ++u) {
                const int ks = (u & 1 ? 3 : 2) << (u >> 1) >> 1;   // 1, 1, 2, 3, 4, 6, 8, .. 48
                if (ks > 1 && ks * 4 > steps) break;
                double t = std::ceil((double)blocks * ks / (cus * c.per_cu)) *
                           (c.fixed + (double)((steps + ks - 1) / ks) * (np == 2 ? c.step2 : c.step3));
                if (ks > 1 || sym) t += 3.5 + (double)I * (double)J * 4.0 * (sym ? 0.5 * ks + 1 : ks + 1) / 4e6;
                if (t < best) { best = t; plan = NsPlan{c.id, ks, sym, (int)blocks}; }
            }
        }
    }
    return plan;
}

struct NsLayout {
    size_t norm, exps, x[2], A, P, partial, total;
    int64_t ldx, ldn, rows;
};
static NsLayout ns_layout(int64_t R, int64_t C, int dt) {
    const size_t np = 3;   // (a 16-bit G may take three pieces)
    const int64_t n = std::min(R, C), m = std::max(R, C);
    NsLayout L{};
    L.rows = R;
    L.ldx = up8(C);
    L.ldn = up8(n);
    size_t off = 0;
    auto take = [&](size_t& at, size_t bytes) { at = off; off = up256(off + bytes); };
    take(L.norm, NORM_WGS * sizeof(double));
    take(L.exps, (ORTHO_MAX_STEPS * NS_EXPS + 2) * sizeof(int));   // (NsExps reads three from any entry)
    for (int i = 0; i < 2; ++i) take(L.x[i], np * (size_t)(R * L.ldx) * 2);
    take(L.A, np * (size_t)(n * L.ldn) * 2);
    take(L.P, np * (size_t)(n * L.ldn) * 2);
    size_t part = 0;
    auto partial = [&](int64_t I, int64_t J, int64_t K, bool symmetric) {
        for (int pieces = dt == DT_F32 ? 3 : 2; pieces <= 3; ++pieces) {
            const NsPlan q = ns_plan(I, J, K, pieces, symmetric);
            if (q.ksplit > 1 || q.sym)
                part = std::max(part, (size_t)q.ksplit * (size_t)(J * ((I + 3) & ~(int64_t)3)) * 4);
        }
    };
    partial(n, n, m, true);
    partial(n, n, n, true);
    partial(C, R, n, false);
    take(L.partial, part);
    L.total = off;
    return L;
}

template <int NP, bool TRU, bool TRV>
static hipError_t ns_product(NsParams p, bool symmetric, hipStream_t s) {
    const NsPlan plan = ns_plan(p.I, p.J, p.K, NP, symmetric);
    p.ksplit = plan.ksplit;
    p.sym = plan.sym;
    auto launch = [&](auto kernel, int ti, int tj, int threads) {
        const int ni = (int)((p.I + ti - 1) / ti), nj = (int)((p.J + tj - 1) / tj);
        hipLaunchKernelGGL(kernel, dim3((unsigned)plan.blocks, (unsigned)p.ksplit), dim3(threads), 0, s, p, ni, nj);
    };
    if constexpr (NP == 2) {
        if (plan.tile == NS_256x128) launch(ns_gemm_kernel<NP, TRU, TRV, 256, 128, 4, 2, 3>, 256, 128, 512);
    }
    if (plan.tile == NS_128x128) launch(ns_gemm_kernel<NP, TRU, TRV, 128, 128, 2, 4, NP == 2 ? 4 : 3>, 128, 128, 512);
    else if (plan.tile == NS_64x64) launch(ns_gemm_kernel<NP, TRU, TRV, 64, 64, 2, 2, 3>, 64, 64, 256);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.sym) {
        const int64_t nb = (p.I + 63) / 64;
        hipLaunchKernelGGL(ns_sym_reduce_kernel<NP>, dim3((unsigned)(nb * (nb + 1) / 2)), dim3(256), 0, s, p);
        e = hipGetLastError();
    } else if (p.ksplit > 1) {
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

    hipLaunchKernelGGL(ns_norm_kernel, dim3(NORM_WGS), dim3(256), 0, s, p.g, p.dt, p.R * p.C,
                       ((uintptr_t)p.g & 15) == 0 ? 1 : 0, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t wgs = std::min<int64_t>((p.R * L.ldx / 8 + 255) / 256, 2048);
    int* const exps = (int*)(W + L.exps);
    SplitParams sp{p.g, p.dt, p.R, p.C, x[0], part, exps, p.steps, p.a, p.b, p.c, p.eps, {}};
    static_assert(ORTHO_MAX_STEPS * NS_EXPS <= 256, "a thread for each of the table");
    ns_exponents<NP>(sp.usual, p.steps, p.a, p.b, p.c, 1.0);
    hipLaunchKernelGGL(ns_split_kernel<NP>, dim3((unsigned)wgs), dim3(256), 0, s, sp);
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
        q.e = exps + k * NS_EXPS;
        q.mode = NS_SPLIT;
        e = tall ? ns_product<NP, true, true>(q, true, s) : ns_product<NP, false, false>(q, true, s);
        if (e != hipSuccess) return e;
        // P = a I + b A + c A A
        q.u = q.v = q.old = A;
        q.o = P;
        q.K = n;
        q.e = exps + k * NS_EXPS + 1;
        q.a = (float)p.a;
        q.b = (float)p.b;
        q.c = (float)p.c;
        q.mode = NS_POLY;
        if ((e = ns_product<NP, false, false>(q, true, s)) != hipSuccess) return e;
        // X <- P X (stored [R][C]: i runs over C, j over R)
        q.e = exps + k * NS_EXPS + 4;
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
            e = ns_product<NP, false, false>(q, false, s);
        } else {
            q.u = cur;
            q.v = P;
            e = ns_product<NP, true, false>(q, false, s);
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

struct ThinLayout {
    size_t part, exps, sum, top, q, fac, chunk_e, x, total;
    int64_t npad, kr, ldx;
    int wgs;
};
static ThinLayout thin_layout(int64_t R, int64_t C) {
    const int64_t n = std::min(R, C), m = std::max(R, C);
    ThinLayout L{};
    L.npad = n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : 128;
    L.kr = std::max<int64_t>(L.npad, 32);
    const int64_t cw = L.npad == 16 ? 256 : L.npad == 32 ? 128 : 64;
    const int64_t chunks = (m + cw - 1) / cw;
    L.ldx = chunks * cw;
    // few enough Gram matrices that adding them up stays short; a long side past
    // 8192 (4096 for 17 .. 32) leaves each workgroup several chunks in turn
    // (bf16 16 x 4096 16 us, 16 x 32768 22, 16 x 131072 40)
    L.wgs = (int)std::min<int64_t>(chunks, L.npad <= 32 ? 32 : 128);
    size_t off = 0;
    auto take = [&](size_t& at, size_t bytes) { at = off; off = up256(off + bytes); };
    take(L.part, (size_t)L.wgs * (size_t)(L.npad * L.npad) * 4);
    take(L.exps, (size_t)L.wgs * 4);
    take(L.sum, (size_t)(L.npad * L.npad) * 4);
    take(L.top, 4);
    take(L.q, 3 * (size_t)(L.npad * L.kr) * 2);
    take(L.fac, 8);
    take(L.chunk_e, (size_t)chunks * 4);
    take(L.x, (size_t)(n * L.ldx) * 4);
    L.total = off;
    return L;
}

template <int NPAD, int NP>
static hipError_t ns_thin(const OrthoParams& p, hipStream_t s) {
    using S = ThinShape<NPAD>;
    const ThinLayout L = thin_layout(p.R, p.C);
    char* W = p.ws;
    ThinParams t{};
    t.g = p.g;
    t.tall = p.R > p.C;
    t.src = t.tall ? 1 : 0;
    t.dt = p.dt;
    t.n = std::min(p.R, p.C);
    t.m = std::max(p.R, p.C);
    t.ldx = L.ldx;
    t.x = (float*)(W + L.x);
    t.q = (const uint16_t*)(W + L.q);
    t.fac = (const double*)(W + L.fac);
    t.part = (float*)(W + L.part);
    t.exps = (int*)(W + L.exps);
    t.chunk_e = (int*)(W + L.chunk_e);
    t.out = p.out;
    t.vec_out = (t.tall ? t.n : t.m) % 4 == 0 && ((uintptr_t)p.out & (p.dt == DT_F32 ? 15 : 7)) == 0;
    t.vec = (t.tall ? t.n : t.m) % 8 == 0 && ((uintptr_t)p.g & 15) == 0;
    // steps a segment: as many as Q's largest factor stays small for (its
    // rounding is relative to it), evenly shared
    constexpr bool WIDE = NPAD == 16 && NP == 2;   // ns_iter64_kernel
    int seg = WIDE ? NS_SEG64 : NP == 2 ? NS_SEG : 1;
    double pall = 1.0, top = 1.0;
    for (int k = 0; k < p.steps; ++k) {
        const NsBounds n = ns_bounds(p.a, p.b, p.c, top);
        pall = std::max(pall, n.p);
        top = n.next;
    }
    while (seg > 1 && std::pow(pall, seg) > NS_QMAX) --seg;
    const int segs = (p.steps + seg - 1) / seg;
    // (ns_loose keeps the bounds below 2^45 and P's above 2^-9; an A or T below
    // 2^-45 loses bits that no P sees)
    auto pow2 = [](double bound) { return std::ldexp(1.f, std::max(-60, std::min(60, ns_exponent<NP>(bound)))); };
    const int64_t chunks = L.ldx / S::CW;
    hipError_t e = hipSuccess;
    top = 1.0;
    int done = 0;
    for (int k = 0; k < segs && e == hipSuccess; ++k) {
        IterParams q{};
        q.part = t.part;
        q.exps = t.exps;
        q.slots = L.wgs;
        q.steps = (p.steps - done + (segs - k) - 1) / (segs - k);
        done += q.steps;
        q.first = k == 0;
        q.a = (float)p.a;
        q.b = (float)p.b;
        q.c = (float)p.c;
        q.eps = p.eps;
        double qmax = 1.0;
        for (int i = 0; i < q.steps; ++i) {
            const NsBounds n = ns_bounds(p.a, p.b, p.c, top);
            qmax *= n.p;
            const int at = WIDE ? 0 : i;   // (the 64-bit segment scales its last Q only)
            q.sA[at] = pow2(top);
            q.sP[at] = pow2(n.p);
            q.sT[at] = pow2(n.lp);
            q.sQ[at] = pow2(qmax);
            top = n.next;
        }
        q.q = (uint16_t*)(W + L.q);
        q.fac = (double*)(W + L.fac);
        // the Gram matrix of X (and X <- Q X of the segment before), then this segment's Q
        if (k == 0) hipLaunchKernelGGL((ns_chunk_kernel<NPAD, NP, THIN_GRAM>), dim3(L.wgs), dim3(S::NT), 0, s, t);
        else hipLaunchKernelGGL((ns_chunk_kernel<NPAD, NP, THIN_BOTH>), dim3(L.wgs), dim3(S::NT), 0, s, t);
        if ((e = hipGetLastError()) != hipSuccess) break;
        if constexpr (NPAD > 32) {
            const int quads = NPAD * NPAD / 4;
            hipLaunchKernelGGL(ns_sum_kernel, dim3(quads / 32), dim3(256), 0, s, t.part, t.exps, L.wgs, quads,
                               (float*)(W + L.sum), (int*)(W + L.top));
            if ((e = hipGetLastError()) != hipSuccess) break;
            q.part = (const float*)(W + L.sum);
            q.exps = (const int*)(W + L.top);
            q.slots = 1;
        }
        if constexpr (WIDE) hipLaunchKernelGGL(ns_iter64_kernel, dim3(1), dim3(64), 0, s, q);
        else hipLaunchKernelGGL((ns_iter_kernel<NPAD, NP>), dim3(1), dim3(iter_threads(NPAD)), 0, s, q);
        if ((e = hipGetLastError()) != hipSuccess) break;
        if (k > 0) {
            t.src = 2;
            t.vec = 1;
        }
    }
    if (e == hipSuccess) {
        hipLaunchKernelGGL((ns_chunk_kernel<NPAD, NP, THIN_OUT>), dim3((unsigned)std::min<int64_t>(chunks, 1024)),
                           dim3(S::NT), 0, s, t);
        e = hipGetLastError();
    }
    return e;
}

// X's exponent follows from what the coefficients can make of |X0|.  Directions
// of small singular values grow by |a| a step, none by more than max |p|: if
// those part by more than 2^8 over the steps, X may be so far below its bound
// that two fp16 pieces lose bits of it (ten are to spare at usual sizes).  So
// are steps that shrink or grow X by 2^9, or A past 2^45: the thin iteration's
// scales and their products stay fp32 numbers.
static bool ns_loose(const OrthoParams& p) {
    double top = 1.0, part = 1.0;
    for (int k = 0; k < p.steps; ++k) {
        const NsBounds n = ns_bounds(p.a, p.b, p.c, top);
        if (n.p < 0x1p-9 || n.p > 0x1p9 || std::max(n.lp, n.next) > 0x1p45) return true;
        part *= n.p / std::fabs(p.a);
        top = n.next;
    }
    return !(part <= 256.0);
}

template <int NP>
static hipError_t ns_run(const OrthoParams& p, hipStream_t s) {
    const int64_t n = std::min(p.R, p.C);
    if (n <= 16) return ns_thin<16, NP>(p, s);
    if (n <= 32) return ns_thin<32, NP>(p, s);
    if (n <= 64) return ns_thin<64, NP>(p, s);
    if (n <= NS_THIN) return ns_thin<128, NP>(p, s);
    return ns_direct<NP>(p, s);
}

OrthoPlan ortho_plan(int64_t R, int64_t C, int dt, int product) {
    const int64_t n = std::min(R, C), m = std::max(R, C);
    if (n <= NS_THIN) return OrthoPlan{0, 0, 0, 0};
    const int np = dt == DT_F32 ? 3 : 2;
    const NsPlan q = product == 0 ? ns_plan(n, n, m, np, true)
                                  : product == 1 ? ns_plan(n, n, n, np, true) : ns_plan(C, R, n, np, false);
    const int tn = q.tile == NS_256x128 ? 256 : q.tile == NS_128x128 ? 128 : 64;
    return OrthoPlan{tn, std::min(tn, 128), q.ksplit, q.sym};
}

size_t ortho_workspace(int64_t R, int64_t C, int dt) {
    if (R <= 0 || C <= 0) return 0;
    return std::min(R, C) <= NS_THIN ? thin_layout(R, C).total : ns_layout(R, C, dt).total;
}

hipError_t launch_ortho(const OrthoParams& p, hipStream_t s) {
    if (p.R <= 0 || p.C <= 0) return hipSuccess;
    return p.dt == DT_F32 || ns_loose(p) ? ns_run<3>(p, s) : ns_run<2>(p, s);
}

}  // namespace lyc
