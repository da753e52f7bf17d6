// fp8gemm.hip -- the product over an 8-bit base weight on gfx950 MFMA:
//
//   y[m][n] = round_out( scale * (h_r . up_c^T)[m][n]
//                        + sum_kb sx[kb][m] * sw[n/128][kb] * sum_{k in kb} qx[m][k] qw[n][k]  + b[n] )
//
// with qx, qw e4m3 codes and one fp32 scale per row group and per weight tile
// of 128.  A K step of the tiles is 128 bytes of every row, exactly one scale
// block: one v_mfma_f32_16x16x128 from a zero accumulator gives the block's
// sum, and one fp32 FMA per element adds it, times the block's two scales, to
// the running sum.  The W side is the MFMA's A operand (a wave's rows share
// one tile scale), the x side its B operand (a lane's column m has one row
// scale), so the product of scales is one value per lane and 16-row block of
// x.
//
// Two instances of the block's sum.  The 8-bit MFMA aligns the products of
// every 8 consecutive k to the largest of them and truncates what lies 13 bits
// below that one's exponent (beside 2^16 it keeps multiples of 2^3; every
// e4m3 MFMA of the device does so; across the groups of 8 it sums in fp32).
// An output is off by up to 7 * 2^-13 of the largest product of each group,
// where nothing cancels less than one step of fp16 and a quarter of bf16's
// rounding, and more where the large ones do; on normal data 1.5e-5 of the result's norm, a
// fourteenth of fp16's rounding and a hundredth of bf16's.  The tiles' 16-bit
// outputs take it for its rate (16384 x 8192 x 1024: 165 us, EXACT 317).  Their
// fp32 outputs, and every output of the few-row kernel, take EXACT: the codes
// widened to fp16, which holds every e4m3 value, and summed by 16-bit MFMAs in
// fp32 at half the rate.
//  The LoRA fold runs first in the same pipeline with 16-bit (or fp32)
// MFMAs, as in gemm.hip.
#include <algorithm>

#include "fp8.h"
#include "gemm_tile.h"
#include "kernels.h"
#include "lyc_device.h"

namespace lyc {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// the sum over one 128-element block: 32 codes of A and of B per lane (bytes
// 16 g .. 16 g + 15 and 64 + 16 g .. of the block for lane group g = lane / 16;
// both sides take the same, so every k meets its own)
__device__ __forceinline__ f32x4 block_dot(i32x4 a0, i32x4 a1, i32x4 b0, i32x4 b1) {
    const i32x8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// 8 codes widened to fp16 (exact)
__device__ __forceinline__ i32x4 widen8(int lo, int hi) {
    i32x4 o;
    o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
    o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
    o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
    o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
    return o;
}

// A block's operand fragment: 32 codes a lane, as loaded or widened
template <bool EXACT>
struct Frag8 {
    i32x4 v[2];
    __device__ __forceinline__ void set(i32x4 a, i32x4 b) { v[0] = a; v[1] = b; }
};
template <>
struct Frag8<true> {
    i32x4 v[4];
    __device__ __forceinline__ void set(i32x4 a, i32x4 b) {
        v[0] = widen8(a[0], a[1]);
        v[1] = widen8(a[2], a[3]);
        v[2] = widen8(b[0], b[1]);
        v[3] = widen8(b[2], b[3]);
    }
};
template <bool EXACT>
__device__ __forceinline__ f32x4 block_sum(const Frag8<EXACT>& a, const Frag8<EXACT>& b) {
    if constexpr (EXACT) {
        f32x4 t = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) t = CF16::step(a.v[i], b.v[i], t);
        return t;
    } else {
        return block_dot(a.v[0], a.v[1], b.v[0], b.v[1]);
    }
}

// A tile whose stages also hold a K step's scales: 64 floats per wave, waves
// 0 .. TM/64-1 the rows' scales, the next wave the tile scales of the TN/128
// (at least one) weight blocks.
template <int TN_, int TM_, int WN_, int WM_, int NS_>
struct Tile8 : Tile<TN_, TM_, WN_, WM_, NS_, 128> {
    using B = Tile<TN_, TM_, WN_, WM_, NS_, 128>;
    static constexpr int DATA = B::STAGE;
    static constexpr int STAGE = DATA + B::NW * 256;
    static constexpr int Q = B::Q + 1;   // loads per wave per step
    static_assert(B::TM / 64 + 1 <= B::NW, "a wave for the tile scales");
    static_assert(NS_ * STAGE + TN_ * 4 <= 160 * 1024, "LDS");
};
using Tile8L = Tile8<256, 256, 128, 64, 2>;
using Tile8M = Tile8<128, 128, 64, 32, 4>;   // 8 waves: with 4, one per SIMD, 777 x 4104 x 4112 took 38 us, not 28
using Tile8S = Tile8<64, 64, 32, 32, 4>;

// ROWS: 16-bit outputs through LDS as whole rows (epilogue_rows).
// 16384 x 8192 x 8192, rank 128: 944 us, 2.4 PFLOP/s (e4m3 MFMA loops with the
// scale FMAs reach 3.3 on random data).  The loads into LDS alone take 746 us,
// MFMAs and FMAs without the fragment reads hide behind them; the reads (192
// of the 256 KiB that go through a CU's LDS each step) do not quite.  Without
// the FMAs, accumulating in the MFMA: 844 us.
template <class CT, class TL, bool ROWS, bool EXACT>
__global__ __launch_bounds__(TL::NT, 1) void fp8_gemm_kernel(Fp8GemmParams pp, int tiles_n, int tiles_m, int group_m) {
    const GemmParams& p = pp.g;
    __shared__ __attribute__((aligned(16))) char smem[TL::NS * TL::STAGE + TL::TN * 4];
    float* sbias = (float*)(smem + TL::NS * TL::STAGE);
    constexpr int FN = TL::FN, FM = TL::FM, NS = TL::NS;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % TL::WAVES_N, wm = wave / TL::WAVES_N;
    int tn, tm;
    tile_coords(blockIdx.x, gridDim.x, tiles_n, tiles_m, group_m, tn, tm);
    const int64_t n0 = (int64_t)tn * TL::TN, m0 = (int64_t)tm * TL::TM;
    const int rows_a = (int)((p.N - n0) < TL::TN ? (p.N - n0) : TL::TN);
    const int rows_b = (int)((p.M - m0) < TL::TM ? (p.M - m0) : TL::TM);

    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // steps: the fold's (with K split 0), then this split's K blocks
    const uint32_t fbytes = (uint32_t)(p.rf * CT::es), kbytes = (uint32_t)p.K;
    const int KM = (int)((kbytes + 127) / 128);
    const int per = (KM + (int)gridDim.y - 1) / (int)gridDim.y;
    const int k0 = (int)blockIdx.y * per;
    const int nmain = KM - k0 < per ? (KM - k0 > 0 ? KM - k0 : 0) : per;
    const int RF = blockIdx.y == 0 ? (int)((fbytes + 127) / 128) : 0;
    const int KT = RF + nmain;
    const char* fa = (const char*)p.af + n0 * fbytes;
    const char* fb = (const char*)p.bf + m0 * fbytes;
    const char* ma = (const char*)p.a + n0 * kbytes;
    const char* mb = (const char*)p.b + m0 * kbytes;
    Loader<TL> lf, lm;
    lf.init(fbytes, fbytes, wave, lane);
    lm.init(kbytes, kbytes, wave, lane);
    // this wave's part of a step's scales (a row's, or a weight tile's)
    const bool is_w = wave == TL::TM / 64;
    const int64_t nblk = (p.N + FP8_BLOCK - 1) / FP8_BLOCK, nb0 = n0 / FP8_BLOCK;
    uint32_t soff = OOB;
    if (wave < TL::TM / 64) {
        if (wave * 64 + lane < rows_b) soff = (uint32_t)(wave * 64 + lane) * 4;
    } else if (is_w) {
        if (lane < (TL::TN + 127) / 128 && nb0 + lane < nblk) soff = (uint32_t)(lane * pp.sw_n) * 4;
    }
    const uint32_t srange = is_w ? (uint32_t)((TL::TN + 127) / 128 * pp.sw_n + 1) * 4 : (uint32_t)rows_b * 4;

    // loads of step s into its stage; past the last step entirely out of range,
    // so that every step issues the same number of loads
    auto issue = [&](int s) {
        char* st = smem + (s % NS) * TL::STAGE;
        const bool fold = s < RF;
        const auto ra = make_rsrc(fold ? fa : ma, (uint32_t)rows_a * (fold ? fbytes : kbytes));
        const auto rb = make_rsrc(fold ? fb : mb, (uint32_t)rows_b * (fold ? fbytes : kbytes));
        Loader<TL> l;
        l.va = fold ? lf.va : lm.va;
        l.vb = fold ? lf.vb : lm.vb;
        l.sa = fold ? lf.sa : lm.sa;
        l.sb = fold ? lf.sb : lm.sb;
        const uint32_t row_bytes = s < KT ? (fold ? fbytes : kbytes) : 0u;
        const int64_t kb = fold ? s : s - RF + k0;
        l.issue(st, ra, rb, row_bytes, (uint32_t)kb * 128u, wave, lane);
        const float* sp = is_w ? pp.sw + nb0 * pp.sw_n + kb * pp.sw_k : pp.sx + kb * p.M + m0;
        const bool on = !fold && s < KT;
        const auto rs = make_rsrc(on ? sp : pp.sw, on ? srange : 0u);
        auto* dst = (__attribute__((address_space(3))) void*)(st + TL::DATA + wave * 256);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst, 4, soff, 0, 0, 0);
    };

    float bv = 0.f;
    if (p.bias != nullptr && p.ksplit <= 1 && tid < TL::TN)
        bv = n0 + tid < p.N ? load_as_f32(p.bias, p.bias_dt, n0 + tid) : 0.f;
    const int g = lane >> 4, r = lane & 15;
#pragma unroll
    for (int s = 0; s < NS; ++s) issue(s);
    if (tid < TL::TN) sbias[tid] = bv;
    wait_vm<(NS - 1) * TL::Q>();
    lds_barrier();
    // Invariant at the head of step kt: its stage has landed for every wave,
    // and the steps up to kt+NS-1 have been issued.  next(kt), once the wave
    // holds all it needs of stage kt in registers: step kt+1 has landed and
    // stage kt is free for step kt+NS.
    auto next = [&]() {
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        wait_vm<(NS - 2) * TL::Q>();
        lds_barrier();
    };
    for (int kt = 0; kt < RF; ++kt) {
        const char* st = smem + (kt % NS) * TL::STAGE;
        const char* sb = st + TL::TN * TL::BKB;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            i32x4 a[FN], b[FM];
#pragma unroll
            for (int i = 0; i < FN; ++i) a[i] = *(const i32x4*)(st + lds_at<TL>(wn * TL::WN + i * 16 + r, sub * 4 + g));
#pragma unroll
            for (int j = 0; j < FM; ++j) b[j] = *(const i32x4*)(sb + lds_at<TL>(wm * TL::WM + j * 16 + r, sub * 4 + g));
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] = CT::step(a[i], b[j], acc[i][j]);
        }
        next();
        issue(kt + NS);
    }
    if (RF > 0) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] *= p.scale;
    }
    const int row_a = wn * TL::WN + r, row_b = wm * TL::WM + r;
    auto load_frag = [&](Frag8<EXACT>& f, const char* base, int row) {
        f.set(*(const i32x4*)(base + lds_at<TL>(row, g)), *(const i32x4*)(base + lds_at<TL>(row, 4 + g)));
    };
    // a step's row scales and this wave's tile scale
    auto load_scales = [&](float (&sj)[FM], const char* st) {
        const float* sc = (const float*)(st + TL::DATA);
#pragma unroll
        for (int j = 0; j < FM; ++j) sj[j] = sc[row_b + j * 16];
        return sc[TL::TM + (wn * TL::WN) / FP8_BLOCK];
    };
    if constexpr (EXACT || FN < 4) {
        for (int kt = RF; kt < KT; ++kt) {
            const char* st = smem + (kt % NS) * TL::STAGE;
            Frag8<EXACT> b[FM];
            float sj[FM];
            const float sw = load_scales(sj, st);
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                load_frag(b[j], st + TL::TN * TL::BKB, row_b + j * 16);
                sj[j] *= sw;
            }
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                Frag8<EXACT> a;
                load_frag(a, st, row_a + i * 16);
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    const f32x4 t = block_sum<EXACT>(a, b[j]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(t[e], sj[j], acc[i][j][e]);
                }
            }
            next();
            issue(kt + NS);
        }
    } else if (KT > RF) {
        // One K step by hand.  A fragments go through a ring of four, read two
        // rows of blocks ahead; a row's MFMAs are followed by the FMAs of the
        // row before, so that the matrix pipe and the vector pipe both have
        // work.  The last two rows of blocks run column by column after the
        // barrier: they need registers only, and each column's B fragment is
        // refilled for the next step as soon as it is used, with a share of
        // the loads of step kt+NS.
        Frag8<false> a[4], b[FM];
        float sj[FM], sn[FM];
        auto fma4 = [&](f32x4& c, const f32x4& t, float sc) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = __builtin_fmaf(t[e], sc, c[e]);
        };
        {
            const char* st = smem + (RF % NS) * TL::STAGE;
            const float sw = load_scales(sj, st);
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                load_frag(b[j], st + TL::TN * TL::BKB, row_b + j * 16);
                sj[j] *= sw;
            }
            load_frag(a[0], st, row_a);
            load_frag(a[1], st, row_a + 16);
        }
        const auto ra = make_rsrc(ma, (uint32_t)rows_a * kbytes);
        const auto rb = make_rsrc(mb, (uint32_t)rows_b * kbytes);
        using LD = Loader<TL>;
        // EARLY (long steps): the wave holds step kt's B fragments and scales in
        // registers from its start, so that side of the stage is released by a
        // barrier of its own and refilled while the A side is still being read:
        // the loads, which bound the step, come in two halves over it
        constexpr bool EARLY = FN > 4;
        constexpr int Q0 = EARLY ? LD::QA : LD::QA + LD::QB;   // loads issued with the last columns
        for (int kt = RF; kt < KT; ++kt) {
            const char* st = smem + (kt % NS) * TL::STAGE;
            const char* nx = smem + ((kt + 1) % NS) * TL::STAGE;
            f32x4 t[2][FM];
            // (steps past the last are out of range; fold steps are all before)
            const int s = kt + NS;
            const int64_t kb = s - RF + k0;
            const uint32_t kb0 = (uint32_t)kb * 128u, row_bytes = s < KT ? kbytes : 0u;
            const bool ok = kb0 + 128u <= row_bytes || kb0 + LD::chunk16(lane) < row_bytes;
            char* wr = smem + (s % NS) * TL::STAGE;
            const float* sp = is_w ? pp.sw + nb0 * pp.sw_n + kb * pp.sw_k : pp.sx + kb * p.M + m0;
            const auto rs = make_rsrc(s < KT ? sp : pp.sw, s < KT ? srange : 0u);
            auto load_side = [&](int q) {   // the q-th of the wave's loads of step kt+NS
                auto* dst = (__attribute__((address_space(3))) void*)(wr + (wave + q * TL::NW) * 1024);
                const bool is_a = q < LD::QA;
                const uint32_t v = is_a ? lm.va + (uint32_t)q * lm.sa : lm.vb + (uint32_t)(q - LD::QA) * lm.sb;
                if (is_a) __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, dst, 16, ok ? v : OOB, (int)kb0, 0, 0);
                else __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, dst, 16, ok ? v : OOB, (int)kb0, 0, 0);
            };
            auto load_scale_row = [&]() {
                auto* dst = (__attribute__((address_space(3))) void*)(wr + TL::DATA + wave * 256);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst, 4, soff, 0, 0, 0);
            };
#pragma unroll
            for (int i = 0; i < FN - 2; ++i) {
                load_frag(a[(i + 2) & 3], st, row_a + (i + 2) * 16);
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    t[i & 1][j] = block_sum<false>(a[i & 3], b[j]);
                    if (i > 0) fma4(acc[i - 1][j], t[(i - 1) & 1][j], sj[j]);
                }
                // an MFMA, then the four FMAs of one column of the row before
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    if (i > 0) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (EARLY && i == 1) {
                    lds_barrier();   // every wave holds its B fragments and scales
#pragma unroll
                    for (int q = LD::QA; q < LD::QA + LD::QB; ++q) load_side(q);
                    load_scale_row();
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            // as next(), the loads in flight counted in the order they go out
            __builtin_amdgcn_s_waitcnt(0xC07F);
            wait_vm<EARLY ? (NS - 1) * (LD::QB + 1) + (NS - 2) * LD::QA : (NS - 2) * TL::Q>();
            lds_barrier();
            const float swn = load_scales(sn, nx);
            load_frag(a[FN & 3], nx, row_a);
            load_frag(a[(FN + 1) & 3], nx, row_a + 16);
            f32x4 u[2][2];
#pragma unroll
            for (int j = 0; j < FM; ++j) {
#pragma unroll
                for (int q = 0; q < Q0; ++q)
                    if (q * FM / Q0 == j) load_side(q);
                u[j & 1][0] = block_sum<false>(a[(FN - 2) & 3], b[j]);
                fma4(acc[FN - 3][j], t[(FN - 3) & 1][j], sj[j]);
                u[j & 1][1] = block_sum<false>(a[(FN - 1) & 3], b[j]);
                if (j > 0) {
                    fma4(acc[FN - 2][j - 1], u[(j - 1) & 1][0], sj[j - 1]);
                    fma4(acc[FN - 1][j - 1], u[(j - 1) & 1][1], sj[j - 1]);
                }
                load_frag(b[j], nx + TL::TN * TL::BKB, row_b + j * 16);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (!EARLY) load_scale_row();
            fma4(acc[FN - 2][FM - 1], u[(FM - 1) & 1][0], sj[FM - 1]);
            fma4(acc[FN - 1][FM - 1], u[(FM - 1) & 1][1], sj[FM - 1]);
#pragma unroll
            for (int j = 0; j < FM; ++j) sj[j] = sn[j] * swn;
            static_assert(FN % 4 == 0, "the ring starts over each step");
        }
    }
    wait_vm<0>();   // the out-of-range loads past the last step still write LDS
    __syncthreads();

    if (p.ksplit > 1) {
        float* part = p.partial + (int64_t)blockIdx.y * p.M * p.N;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int64_t nb = n0 + wn * TL::WN + i * 16 + 4 * g;
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const int64_t m = m0 + wm * TL::WM + j * 16 + r;
                if (m >= p.M) continue;
                float* dst = part + m * p.N + nb;
                if (p.vec_store && nb + 3 < p.N) {
                    *(f32x4*)dst = acc[i][j];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nb + e < p.N) dst[e] = acc[i][j][e];
                }
            }
        }
        return;
    }
    float biasv[FN * 4] = {};
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        const f32x4 b4 = *(const f32x4*)(sbias + wn * TL::WN + i * 16 + 4 * g);
        biasv[4 * i] = b4[0]; biasv[4 * i + 1] = b4[1]; biasv[4 * i + 2] = b4[2]; biasv[4 * i + 3] = b4[3];
    }
    if constexpr (ROWS) {
        epilogue_rows<TL, 2, false>(p, smem, acc, biasv, biasv, n0, m0, wave, lane, wn, wm);
        return;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        const int64_t nb = n0 + wn * TL::WN + i * 16 + 4 * g;
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int64_t m = m0 + wm * TL::WM + j * 16 + r;
            if (m >= p.M) continue;
            if (p.y_dt == DT_F32 && p.vec_store && nb + 3 < p.N) {
                f32x4 v = acc[i][j];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += biasv[4 * i + e];
                *(f32x4*)((float*)p.y + m * p.N + nb) = v;
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = acc[i][j][e] + biasv[4 * i + e];
                if (nb + e >= p.N) continue;
                const int64_t at = m * p.N + nb + e;
                if (p.y_dt == DT_F32) ((float*)p.y)[at] = v;
                else ((uint16_t*)p.y)[at] = p.y_dt == DT_F16 ? f32_to_f16(v) : f32_to_bf16(v);
            }
        }
    }
}

// ---- few token rows: one workgroup per 16 NF output features ----------------------
// All of K in one workgroup, wave w of the NW taking the w-th share of the
// 128-byte blocks, its fragments and scales read straight from global memory D
// blocks ahead (every weight byte is used once); the waves' sums meet in LDS
// in wave order, wave 0's with the fold.  Bound by the weight's bytes: x's
// rows, read by every workgroup from L2, cost as much again per 16 features,
// so NF = 2 where that still leaves a workgroup per CU.  The matrix pipe has
// room, so the codes are widened and the sums are fp32 throughout: 14.5 us at
// 16 x 8192 x 8192 where 8-bit MFMAs took 14.4, 56.7 for 54.8 at 16 x 28672 x 8192.
template <class CT, int MT, int NF, int D, int NW>
__global__ __launch_bounds__(64 * NW) void fp8_skinny_kernel(Fp8GemmParams pp) {
    const GemmParams& p = pp.g;
    __shared__ __attribute__((aligned(16))) f32x4 red[NW][NF][MT][64];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NF);
    const uint32_t kb = (uint32_t)p.K;
    const int nrows = (int)(p.N - n0 < 16 * NF ? p.N - n0 : 16 * NF);
    const auto rw = make_rsrc_uniform((const char*)p.a + n0 * kb, (uint32_t)nrows * kb);
    const auto rx = make_rsrc_uniform(p.b, (uint32_t)p.M * kb);
    const int blocks = (int)((kb + 127) / 128);
    const auto rs = make_rsrc_uniform(pp.sx, (uint32_t)(blocks * p.M) * 4);
    const float* sw = pp.sw + n0 / FP8_BLOCK * pp.sw_n;   // (16 NF features lie in one tile)
    f32x4 acc[NF][MT];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (wave == 0 && p.rf > 0) {
        const uint32_t fb = (uint32_t)(p.rf * CT::es), lo = (uint32_t)g * 16;
        const auto ru = make_rsrc_uniform((const char*)p.af + n0 * fb, (uint32_t)nrows * fb);
        const auto rh = make_rsrc_uniform(p.bf, (uint32_t)p.M * fb);
        for (uint32_t k = 0; k < fb; k += 64) {
            i32x4 hb[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) hb[t] = buf_load16(rh, k + lo < fb ? (uint32_t)(16 * t + r) * fb + k + lo : OOB);
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const i32x4 ua = buf_load16(ru, k + lo < fb ? (uint32_t)(16 * f + r) * fb + k + lo : OOB);
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[f][t] = CT::step(ua, hb[t], acc[f][t]);
            }
        }
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[f][t] *= p.scale;
    }

    // ring slot u holds block s0 + u (mod D); past the share's end everything
    // is sent out of range and reads zeros
    const int s0 = blocks * wave / NW, s1 = blocks * (wave + 1) / NW;
    const int se = s0 + ((s1 - s0 + D - 1) / D) * D;
    i32x4 wa[D][NF][2], xa[D][MT][2];
    float sx[D][MT], sv[D];
    auto load = [&](int u, int b) {
        const bool on = b < s1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t k = (uint32_t)b * 128 + (uint32_t)(h * 64 + g * 16);
            const bool in = on && k < kb;
#pragma unroll
            for (int f = 0; f < NF; ++f) wa[u][f][h] = buf_load16(rw, in ? (uint32_t)(16 * f + r) * kb + k : OOB);
#pragma unroll
            for (int t = 0; t < MT; ++t) xa[u][t][h] = buf_load16(rx, in ? (uint32_t)(16 * t + r) * kb + k : OOB);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
            sx[u][t] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                rs, on && 16 * t + r < p.M ? (uint32_t)(b * p.M + 16 * t + r) * 4 : OOB, 0, 0));
        sv[u] = sw[(on ? b : 0) * pp.sw_k];
    };
#pragma unroll
    for (int u = 0; u < D; ++u) load(u, s0 + u);
    for (int sb = s0; sb < se; sb += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            Frag8<true> fx[MT];
            float sc[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                fx[t].set(xa[u][t][0], xa[u][t][1]);
                sc[t] = sx[u][t] * sv[u];
            }
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                Frag8<true> fw;
                fw.set(wa[u][f][0], wa[u][f][1]);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const f32x4 v = block_sum<true>(fw, fx[t]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[f][t][e] = __builtin_fmaf(v[e], sc[t], acc[f][t][e]);
                }
            }
            load(u, sb + u + D);
        }
    }
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int t = 0; t < MT; ++t) red[wave][f][t][lane] = acc[f][t];
    __syncthreads();
    static_assert(NF * MT <= NW, "a wave per output block");
    // wave w < NF MT adds up and stores block (f, t) = (w / MT, w % MT)
    if (wave >= NF * MT) return;
    const int f = wave / MT, t = wave % MT;
    f32x4 sum = red[0][f][t][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += red[w][f][t][lane];
    const int64_t nb = n0 + 16 * f + 4 * g, m = 16 * t + r;
    if (m >= p.M) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (nb + e >= p.N) continue;
        const float v = sum[e] + (p.bias != nullptr ? load_as_f32(p.bias, p.bias_dt, nb + e) : 0.f);
        const int64_t at = m * p.N + nb + e;
        if (p.y_dt == DT_F32) ((float*)p.y)[at] = v;
        else ((uint16_t*)p.y)[at] = p.y_dt == DT_F16 ? f32_to_f16(v) : f32_to_bf16(v);
    }
}

// the few-row kernel's limits: 32 rows, 32-bit offsets
static bool fp8_skinny(int64_t M, int64_t K) {
    return M >= 1 && M <= 32 && K > 0 && 32 * K < ((int64_t)1 << 31);
}

// enough features for a workgroup per CU at 32 each
static bool fp8_wide(int64_t N) { return N >= 32 * device_rates().cus; }

template <class CT, int MT, int NF>
static hipError_t run_skinny8(const Fp8GemmParams& p, hipStream_t s) {
    // 4 waves, 2 blocks ahead: more waves or loads in flight were slower (16 x
    // 8192 x 8192: 14.6 us; 8 waves 19.4, 4 blocks ahead 15.0, 8 ahead 15.8)
    hipLaunchKernelGGL((fp8_skinny_kernel<CT, MT, NF, 2, 4>), dim3((unsigned)((p.g.N + 16 * NF - 1) / (16 * NF))),
                       dim3(256), 0, s, p);
    return hipGetLastError();
}
template <class CT>
static hipError_t run_skinny8_ct(const Fp8GemmParams& p, hipStream_t s) {
    const bool wide = fp8_wide(p.g.N);
    if (p.g.M <= 16) return wide ? run_skinny8<CT, 1, 2>(p, s) : run_skinny8<CT, 1, 1>(p, s);
    return wide ? run_skinny8<CT, 2, 2>(p, s) : run_skinny8<CT, 2, 1>(p, s);
}

enum { T8_L, T8_M, T8_S };

// Output tile and K split by modelled time, us: rounds of workgroups over the
// CUs (two 64 x 64 ones share one), each a fixed part and its K steps, plus a
// split's partial sums out and in again.  Measured steps of 128, on a device
// up to four fifths full (64 x 64: of one a CU) and full:
//             16-bit y (8-bit MFMAs)      fp32 y (EXACT)
//   256 x 256    1.3, 1.3  fixed 10.5       3.05, 3.05  fixed 12
//   128 x 128    0.41, 0.5       7          1.1, 1.1          6
//   64 x 64      0.42, 0.52      5          0.57, 0.8         5
// (16-bit rows of y that are not whole 16-byte pieces are stored by element: 15,
// 4.5 and 1.5 more: 2500 x 2500 x 2560 took 50.0 in 256 x 256, 2560 x 2560 34.3.)
// Whole calls, the pick and what it is held against: 64 x 4096 x 4096 bf16 64 x
// 64 tiles in 4 splits 12.0, one 17.6; 1024 x 1024 x 8192 bf16 128 x 128 in 4
// splits 22.5, 64 x 64 in one 32.0; 256 x 2048 x 4096 fp32 64 x 64 in 4 splits
// 15.8, in one 23.3.
static void fp8_pick(int64_t M, int64_t N, int64_t K, bool exact, int* tile, int* ksplit) {
    struct C { int id, tn, tm, per_cu; double light, fixed, few, full, by_element; };
    const C cands[2][3] = {
        {{T8_L, 256, 256, 1, 0.8, 10.5, 1.3, 1.3, 15.0},
         {T8_M, 128, 128, 1, 0.8, 7.0, 0.41, 0.5, 4.5},
         {T8_S, 64, 64, 2, 1.0, 5.0, 0.42, 0.52, 1.5}},
        {{T8_L, 256, 256, 1, 0.8, 12.0, 3.05, 3.05, 0.0},
         {T8_M, 128, 128, 1, 0.8, 6.0, 1.1, 1.1, 0.0},
         {T8_S, 64, 64, 2, 1.0, 5.0, 0.57, 0.8, 0.0}}};
    const double cus = (double)device_rates().cus;
    const int64_t ksteps = (K + 127) / 128;
    double best = 1e300;
    *tile = T8_S;
    *ksplit = 1;
    for (const C& c : cands[exact ? 1 : 0]) {
        const double tiles = (double)((N + c.tn - 1) / c.tn) * (double)((M + c.tm - 1) / c.tm);
        for (int ks = 1; ks <= 8; ks *= 2) {
            if (ks > 1 && (ks > ksteps / 2 || (double)M * N * 4.0 * ks > 32.0 * 1024 * 1024)) continue;
            const double steps = (double)((ksteps + ks - 1) / ks);
            const double fixed = c.fixed + (ks == 1 && N % 8 != 0 ? c.by_element : 0.0);
            const double rounds = std::ceil(tiles * ks / (cus * c.per_cu));
            double t = rounds * (fixed + steps * (tiles * ks <= c.light * rounds * cus ? c.few : c.full));
            if (ks > 1) t += 2.5 + (double)M * N * 4.0 * (ks + 1) / 2.5e6;
            if (t < best) { best = t; *tile = c.id; *ksplit = ks; }
        }
    }
}

Fp8Plan fp8_gemm_plan(int64_t M, int64_t N, int64_t K, int y_dt) {
    if (M <= 0 || N <= 0) return Fp8Plan{0, 0, 1};
    if (fp8_skinny(M, K)) return Fp8Plan{fp8_wide(N) ? 32 : 16, M <= 16 ? 16 : 32, 1};
    int t, ks;
    fp8_pick(M, N, K, y_dt == DT_F32, &t, &ks);
    const int tn = t == T8_L ? 256 : t == T8_M ? 128 : 64;
    return Fp8Plan{tn, tn, ks};
}

template <class CT, class TL>
static hipError_t run8(const Fp8GemmParams& p, hipStream_t s) {
    const int64_t tiles_n = (p.g.N + TL::TN - 1) / TL::TN, tiles_m = (p.g.M + TL::TM - 1) / TL::TM;
    if (tiles_n * tiles_m >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    const int ks = p.g.ksplit > 1 ? p.g.ksplit : 1;
    const dim3 grid((unsigned)(tiles_n * tiles_m), ks);
    const bool rows = ks == 1 && (p.g.N * 2) % 16 == 0 && ((uintptr_t)p.g.y & 15) == 0;
    if (p.g.y_dt == DT_F32) {
        hipLaunchKernelGGL((fp8_gemm_kernel<CT, TL, false, true>), grid, dim3(TL::NT), 0, s, p, (int)tiles_n,
                           (int)tiles_m, 4);
    } else if constexpr (CT::dt == DT_F32) {
        return hipErrorInvalidValue;   // fp32 compute gives fp32 outputs
    } else if (rows) {
        hipLaunchKernelGGL((fp8_gemm_kernel<CT, TL, true, false>), grid, dim3(TL::NT), 0, s, p, (int)tiles_n,
                           (int)tiles_m, 4);
    } else {
        hipLaunchKernelGGL((fp8_gemm_kernel<CT, TL, false, false>), grid, dim3(TL::NT), 0, s, p, (int)tiles_n,
                           (int)tiles_m, 4);
    }
    if (ks > 1) {
        const hipError_t e = hipGetLastError();
        return e != hipSuccess ? e : launch_gemm_reduce(p.g, s);
    }
    return hipGetLastError();
}

template <class CT>
static hipError_t run8_ct(const Fp8GemmParams& p, int t, hipStream_t s) {
    if (t == T8_L) return run8<CT, Tile8L>(p, s);
    if (t == T8_M) return run8<CT, Tile8M>(p, s);
    return run8<CT, Tile8S>(p, s);
}

hipError_t launch_fp8_gemm(int c_dt, const Fp8GemmParams& p, hipStream_t s) {
    if (p.g.M <= 0 || p.g.N <= 0) return hipSuccess;
    if (p.g.ksplit <= 1 && fp8_skinny(p.g.M, p.g.K)) {
        if (c_dt == DT_F16) return run_skinny8_ct<CF16>(p, s);
        if (c_dt == DT_BF16) return run_skinny8_ct<CBF16>(p, s);
        return run_skinny8_ct<CF32>(p, s);
    }
    int t, ks;
    fp8_pick(p.g.M, p.g.N, p.g.K, p.g.y_dt == DT_F32, &t, &ks);
    if (p.g.ksplit > 1 && p.g.partial == nullptr) return hipErrorInvalidValue;
    if (c_dt == DT_F16) return run8_ct<CF16>(p, t, s);
    if (c_dt == DT_BF16) return run8_ct<CBF16>(p, t, s);
    return run8_ct<CF32>(p, t, s);
}

}  // namespace lyc
