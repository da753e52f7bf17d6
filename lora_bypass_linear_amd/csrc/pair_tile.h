// pair_tile.h -- the tiled MFMA products of the gated feed-forward block and of
// the 8-bit integers (pair.h says what each mode computes).
//
// One workgroup owns one output tile.  In PAIR mode the A side of the tile
// interleaves the two weights: of every WN rows that one wave multiplies, the
// first half are rows of a[0] and the second half the same features' rows of
// a[1], so a lane holds g and v of the same outputs in its own registers and
// the block's two projections, its activation and its product are one kernel:
// g and v (M x N each) never reach memory unless they are kept.  A K step costs
// what a step of one product with 2 N features costs.
//
// K steps come in segments: the folds (PAIR, SEQ: one per factor pair), then
// the contraction over K (SEQ: one after the other).  A feed keeps the
// position of the next load: its pointers, ranges and row strides are uniform
// values that change between segments only.
//
// int8 sums are exact 32-bit integers (127^2 K < 2^31), so neither the order of
// the K steps nor a K split changes a result; they become fp32 once, at the end.
//
// fp32 products are summed in blocks of SUM_K: one chain of n fused steps is off
// by about sqrt(n / 2) 2^-25 of the result (independent terms, partial sums that
// grow as sqrt(k)), n / b blocks of b by sqrt(b / 2 + n / 2b) 2^-25.  (16-bit
// products enter the chain 32 at a time, so theirs is short.)  20 x 512 x 8192:
// 1.1e-6 of the norm as chains of 2048, 5.6e-7 so, in the same time.
//
// What bounds it: at the large sizes the matrix pipe (busy about 65 % of the
// cycles, clocked down under its load) with the stream of operands from L2 into
// LDS behind it: a 256 x 256 step takes 1.4 us, its loads alone 1.1, its MFMAs
// alone 0.9.  int8 16384 x 8192 x 8192: 823-842 us, 2.6 POP/s; bf16 block 8192 x 8192 x
// 4096 rank 64 with g and v kept: about 865 us, 1.3 PFLOP/s.  Eight waves of 128 x 64 and
// not four of 128 x 128: their accumulators fill the AGPRs, and the compiler moves
// them every step.  Two stages of 128-byte steps and not four of 64 (845 against
// 880 us).  Few rows: pair_skinny_kernel below, bound by the weights' bytes.
#pragma once

#include <type_traits>

#include "act.h"
#include "gemm_tile.h"
#include "lyc_device.h"
#include "pair.h"

namespace lyc {

struct CI8 {
    static constexpr int dt = DT_I8;
    static constexpr int es = 1;
    // v_mfma_i32_16x16x64_i8: a lane's 16 bytes are 16 k values, the output
    // layout that of the 16-bit forms
    __device__ static __forceinline__ i32x4 step(i32x4 a, i32x4 b, i32x4 c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
};
template <class CT>
using Acc = std::conditional_t<CT::dt == DT_I8, i32x4, f32x4>;

constexpr int SUM_K = 512;   // products of a block of an fp32 sum

__device__ __forceinline__ f32x4 to_f32(f32x4 v) { return v; }
__device__ __forceinline__ f32x4 to_f32(i32x4 v) { return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]}; }

// body(act): one copy of the caller's loop for each form of the activation, the
// choice (uniform) outside it; WIDE: for fp32 results
template <bool WIDE, class F>
__device__ __forceinline__ void with_activation(int act, F body) {
    if (act == ACT_GELU) {
        body([](float g) { return act_gelu<false>(g, nullptr, nullptr); });
    } else {
        float a, b;
        act_coeffs(act, a, b);
        if constexpr (WIDE) body([=](float g) { return act_logistic<false>(a, b, g, nullptr); });
        else body([=](float g) { return act_logistic16(a, b, g); });
    }
}

// 16 bytes at any address
struct __attribute__((packed)) Any16 {
    i32x4 v;
};

template <class TL, int MODE>
struct PairShape {
    static constexpr bool TWO = MODE == PAIR_PAIR;
    static constexpr int TF = TWO ? TL::TN / 2 : TL::TN;   // features of the tile
    static constexpr int WF = TWO ? TL::WN / 2 : TL::WN;   // of a wave
    static constexpr int FI = TWO ? TL::FN / 2 : TL::FN;   // 16-feature blocks of a wave
    static_assert(!TWO || WF % 16 == 0, "a wave's two halves");
};

// The position of the next K step's loads
template <class CT, class TL, int MODE>
struct Feed {
    using SH = PairShape<TL, MODE>;
    static constexpr int QA = TL::TN / TL::RPB / TL::NW, QB = TL::TM / TL::RPB / TL::NW;
    static_assert(QA * TL::RPB * TL::NW == TL::TN && QB * TL::RPB * TL::NW == TL::TM, "loader split");
    static_assert(TL::BKB == 128, "8 rows a wave load");
    const char *pa0, *pa1, *pb;    // the tile's rows of this segment
    uint32_t na0, na1, nb;         // their byte extents (buffer range; 0: reads zeros)
    uint32_t row;                  // valid bytes of a row in this segment
    uint32_t kb0;                  // first byte of the next step within a row
    uint32_t sa, sb;               // row strides in bytes
    uint32_t va, vb;               // lane offsets of its first A / B block at step 0
    int left, seg, k0, nmain;      // steps left in the segment; K split's main steps
    bool folds;

    // byte chunk of a row that the lane fetches (the swizzle of lds_at)
    __device__ __forceinline__ static uint32_t chunk(int lane) { return (uint32_t)((lane & 7) ^ (lane >> 3)) << 4; }

    __device__ __forceinline__ void enter(const PairParams& p, int64_t n0, int64_t m0, int rows_a, int rows_b, int wave,
                                          int lane) {
        const bool fold = seg < 2;
        const int h = seg & 1;
        const uint32_t ka = (uint32_t)((fold ? p.rf : p.K) * CT::es);
        sa = ka;
        sb = fold ? (uint32_t)(p.ldf * CT::es) : ka;
        row = ka;
        const void* a0 = fold ? (h ? p.af[1] : p.af[0]) : (h && !SH::TWO ? p.a[1] : p.a[0]);
        const void* bq = fold ? (h ? p.bf[1] : p.bf[0]) : (h && !SH::TWO ? p.b[1] : p.b[0]);
        const uint32_t ext = (uint32_t)rows_a * ka;
        pa0 = (const char*)a0 + n0 * ka;
        na0 = ext;
        if constexpr (SH::TWO) {
            // a fold step multiplies one factor pair: the other half's rows, which take no
            // part in it, read zeros (every step issues the same loads)
            pa1 = fold ? pa0 : (const char*)p.a[1] + n0 * ka;
            na1 = fold && h == 0 ? 0u : ext;
            na0 = fold && h == 1 ? 0u : ext;
        } else {
            pa1 = pa0;
            na1 = na0;
        }
        pb = (const char*)bq + m0 * sb;
        nb = (uint32_t)(rows_b - 1) * sb + ka;
        kb0 = fold ? 0u : (uint32_t)k0 * TL::BKB;
        left = fold ? (int)((ka + TL::BKB - 1) / TL::BKB) : nmain;
        const uint32_t l8 = (uint32_t)(lane >> 3);
        vb = ((uint32_t)(wave * 8) + l8) * sb + chunk(lane);
        va = l8 * sa + chunk(lane);
    }
    __device__ __forceinline__ void stop() {
        row = 0;
        left = 1 << 30;
    }
    // to the next segment that has steps; past the last one every load is out
    // of range (it writes zeros into a stage that is never read), so that each
    // step issues the same number of loads
    __device__ __forceinline__ void next_segment(const PairParams& p, int64_t n0, int64_t m0, int rows_a, int rows_b,
                                                 int wave, int lane) {
        constexpr int LAST = MODE == PAIR_SEQ ? 3 : 2;
        for (;;) {
            ++seg;
            if (seg < 2 && !folds) seg = 2;
            if (seg > LAST) {
                stop();
                return;
            }
            enter(p, n0, m0, rows_a, rows_b, wave, lane);
            if (left > 0) return;
        }
    }
    // first tile row, and which matrix, of the wave's q-th A block
    __device__ __forceinline__ static void a_block(int wave, int q, int& half, int& feature) {
        if constexpr (!SH::TWO) {
            half = 0;
            feature = 8 * (wave + q * TL::NW);
        } else if constexpr (TL::NW * 8 == SH::WF) {
            half = q & 1;
            feature = (q >> 1) * SH::WF + 8 * wave;
        } else {
            const int r0 = 8 * (wave + q * TL::NW);
            half = (r0 % TL::WN) / SH::WF;
            feature = (r0 / TL::WN) * SH::WF + r0 % SH::WF;
        }
    }
    // the wave's q-th load of the next step into stage st (q < QA: A side)
    __device__ __forceinline__ void load(int q, char* st, bool ok, int wave) const {
        auto* dst = (__attribute__((address_space(3))) void*)(st + (wave + q * TL::NW) * 1024);
        if (q < QA) {
            int half, f;
            a_block(wave, q, half, f);
            const uint32_t v = va + (uint32_t)f * sa;
            const char* pa = half ? pa1 : pa0;
            const uint32_t na = half ? na1 : na0;
            const auto ra = make_rsrc(pa, na);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, dst, 16, ok ? v : OOB, (int)kb0, 0, 0);
        } else {
            const auto rb = make_rsrc(pb, nb);
            const uint32_t v = vb + (uint32_t)((q - QA) * TL::NW * 8) * sb;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, dst, 16, ok ? v : OOB, (int)kb0, 0, 0);
        }
    }
    __device__ __forceinline__ bool ok(int lane) const {
        return kb0 + TL::BKB <= row || kb0 + chunk(lane) < row;
    }
};

// One tile's outputs of one tensor through LDS, so that every store writes
// whole rows of it (a lane's results are 4 features of one token; stored
// directly they would be 8- to 16-byte pieces of 16 rows).  val(i, j) gives the
// lane's 4 values of block (i, j).  Rows start at any element boundary: the
// 16-byte stores need no alignment, and a row's last, partial chunk goes out by
// element.
template <class TL, int MODE, int ES, class F>
__device__ __forceinline__ void store_tile(char* smem, F val, void* y, int y_dt, int64_t M, int64_t N, int64_t n0,
                                           int64_t m0, int wave, int lane, int wn, int wm) {
    using SH = PairShape<TL, MODE>;
    // (chunks are permuted within a row by its low bits, 8 or 4 of them)
    constexpr int RB = SH::TF * ES, CHR = RB / 16, SW = CHR % 8 == 0 ? 7 : 3;
    static_assert(CHR % 4 == 0, "permuted chunks");
    constexpr int CAP = TL::NS * TL::STAGE;
    constexpr int TMP = TL::TM * RB <= CAP ? TL::TM : TL::TM / 2;   // rows per pass
    constexpr int PASSES = TL::TM / TMP, IT = TMP * CHR / TL::NT;
    static_assert(TMP * RB <= CAP && TMP % TL::WM == 0 && IT * TL::NT == TMP * CHR, "staged rows");
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        if ((wm * TL::WM) / TMP == ps) {
#pragma unroll
            for (int i = 0; i < SH::FI; ++i) {
                const int cb = (wn * SH::WF + i * 16 + 4 * (lane >> 4)) * ES;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < TL::FM; ++j) {
                    const int r = wm * TL::WM + j * 16 + (lane & 15) - ps * TMP;
                    const f32x4 v = val(i, j);
                    char* dst = smem + r * RB + ((((cb >> 4) ^ (r & SW)) << 4) | (cb & 15));
                    if constexpr (ES == 4) {
                        *(f32x4*)dst = v;
                    } else {
                        const uint32_t lo = y_dt == DT_F16 ? pack_f16x2(v[0], v[1]) : pack_bf16x2(v[0], v[1]);
                        const uint32_t hi = y_dt == DT_F16 ? pack_f16x2(v[2], v[3]) : pack_bf16x2(v[2], v[3]);
                        *(i32x2*)dst = i32x2{(int)lo, (int)hi};
                    }
                }
            }
        }
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll 4
        for (int it = 0; it < IT; ++it) {
            const int idx = (it * TL::NW + wave) * 64 + lane;
            const int r = idx / CHR, c = idx % CHR;
            const i32x4 d = *(const i32x4*)(smem + r * RB + ((c ^ (r & SW)) << 4));
            const int64_t m = m0 + ps * TMP + r, n = n0 + c * (16 / ES);
            if (m >= M || n >= N) continue;
            char* dst = (char*)y + (m * N + n) * ES;
            if (n + 16 / ES <= N) {
                ((Any16*)dst)->v = d;
            } else {
                const int left = (int)(N - n);
#pragma unroll
                for (int e = 0; e < 16 / ES; ++e) {
                    if (e >= left) continue;
                    if constexpr (ES == 4) ((int*)dst)[e] = d[e];
                    else ((uint16_t*)dst)[e] = (uint16_t)((uint32_t)d[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
    }
}

template <class CT, class TL, int MODE>
__global__ __launch_bounds__(TL::NT, 1) void pair_kernel(PairParams p, int tiles_n, int tiles_m, int group_m) {
    using SH = PairShape<TL, MODE>;
    using FD = Feed<CT, TL, MODE>;
    constexpr bool I8 = CT::dt == DT_I8;
    constexpr int FN = TL::FN, FM = TL::FM, NS = TL::NS, Q = TL::Q;
    // the operand stages, then biases (TN), int8: the weights' scales (TN) and x's (TM).
    // One LDS object: with a second one the compiler cannot tell the
    // direct-to-LDS loads from the fragment reads and waits for every load.
    __shared__ __attribute__((aligned(16))) char smem[NS * TL::STAGE + (I8 ? 2 * TL::TN + TL::TM : TL::TN) * 4];
    float* aux = (float*)(smem + NS * TL::STAGE);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % TL::WAVES_N, wm = wave / TL::WAVES_N;
    int tn, tm;
    tile_coords(blockIdx.x, gridDim.x, tiles_n, tiles_m, group_m, tn, tm);
    const int64_t n0 = (int64_t)tn * SH::TF, m0 = (int64_t)tm * TL::TM;
    const int rows_a = (int)((p.N - n0) < SH::TF ? (p.N - n0) : SH::TF);
    const int rows_b = (int)((p.M - m0) < TL::TM ? (p.M - m0) : TL::TM);

    Acc<CT> acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = Acc<CT>{};

    FD fd;
    const int KM = (int)((p.K * CT::es + TL::BKB - 1) / TL::BKB);
    const int per = (KM + (int)gridDim.y - 1) / (int)gridDim.y;
    fd.k0 = (int)blockIdx.y * per;
    fd.nmain = KM - fd.k0 < per ? (KM - fd.k0 > 0 ? KM - fd.k0 : 0) : per;
    fd.folds = !I8 && p.rf > 0 && blockIdx.y == 0;
    fd.seg = -1;
    const int RF = fd.folds ? 2 * (int)((p.rf * CT::es + TL::BKB - 1) / TL::BKB) : 0;
    const int KT = RF + (MODE == PAIR_SEQ ? 2 : 1) * fd.nmain;

    // loaded ahead of the operands, written to LDS behind their issue
    float bv = 0.f, sw = 0.f, sx = 0.f;
    if (p.ksplit <= 1 && tid < TL::TN) {
        const int half = SH::TWO ? tid / SH::TF : 0;
        const int64_t n = n0 + (SH::TWO ? tid % SH::TF : tid);
        const void* bp = half ? p.bias[1] : p.bias[0];
        if (n < p.N) {
            if (bp != nullptr) bv = load_as_f32(bp, p.bias_dt, n);
            if (I8) sw = (half ? p.sw[1] : p.sw[0])[n];
        }
    }
    if (I8 && p.ksplit <= 1 && tid < rows_b) sx = p.sx[m0 + tid];

    if (KT > 0) {
        i32x4 f0a[FN], f0b[FM], f1a[FN], f1b[FM];
        fd.next_segment(p, n0, m0, rows_a, rows_b, wave, lane);
        auto advance = [&]() {
            fd.kb0 += TL::BKB;
            if (--fd.left == 0) fd.next_segment(p, n0, m0, rows_a, rows_b, wave, lane);
        };
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const bool ok = fd.ok(lane);
#pragma unroll
            for (int q = 0; q < FD::QA + FD::QB; ++q) fd.load(q, smem + s * TL::STAGE, ok, wave);
            advance();
        }
        const int r = lane & 15, g4 = lane >> 4;
        auto frag_a = [&](const char* st, int sub, int i) {
            return *(const i32x4*)(st + lds_at<TL>(wn * TL::WN + i * 16 + r, sub * 4 + g4));
        };
        auto frag_b = [&](const char* st, int sub, int j) {
            return *(const i32x4*)(st + TL::TN * TL::BKB + lds_at<TL>(wm * TL::WM + j * 16 + r, sub * 4 + g4));
        };
        wait_vm<(NS - 1) * Q>();
        lds_barrier();
#pragma unroll
        for (int i = 0; i < FN; ++i) f0a[i] = frag_a(smem, 0, i);
#pragma unroll
        for (int j = 0; j < FM; ++j) f0b[j] = frag_b(smem, 0, j);

        // One K step (two MFMA substeps of 64 bytes).  Substep 0's fragments are
        // in registers on entry; substep 1's are read under its MFMAs.  The
        // first MFMAs of substep 1 are issued before the wait for step kt+1 and
        // the barrier; after it the loads of step kt+NS into the stage just
        // consumed and the next fragments go between the others.
        // A fold step of the gated block belongs to one projection: only that one's
        // blocks (HALF 0 or 1) take part, since zeros for the other's rows would turn
        // an h that is not finite into NaNs there (HALF 2: every block).
        auto k_step = [&](int kt, auto half) {
            constexpr int HALF = decltype(half)::value;
            constexpr int I0 = HALF == 1 ? SH::FI : 0, I1 = HALF == 0 ? SH::FI : FN;
            constexpr int ND = FN + FM;
            constexpr int G = FN % 4 == 0 ? 4 : 2, FNG = FN / G;
            char* st = smem + (kt % NS) * TL::STAGE;
            __builtin_amdgcn_s_waitcnt(0xC07F);
#pragma unroll
            for (int i = 0; i < FN; ++i) f1a[i] = frag_a(st, 1, i);
#pragma unroll
            for (int j = 0; j < FM; ++j) f1b[j] = frag_b(st, 1, j);
#pragma unroll
            for (int i = I0; i < I1; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] = CT::step(f0a[i], f0b[j], acc[i][j]);
            constexpr int NF = (I1 - I0) * FM, PER = NF / (ND + 1);
            if constexpr (PER > 0) {
#pragma unroll
                for (int g = 0; g < ND; ++g) {
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x008, NF - ND * PER, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);
#pragma unroll
            for (int i = 0; i < FNG; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    if (i >= I0 && i < I1) acc[i][j] = CT::step(f1a[i], f1b[j], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
            wait_vm<(NS - 2) * Q>();
            lds_barrier();
            const bool ok = fd.ok(lane);
            const char* nx = smem + ((kt + 1) % NS) * TL::STAGE;
            // Q slots of a load, a share of the fragment reads (done three quarters
            // through) and of the MFMAs.  A load occupies the CU's address path for
            // 16 cycles: issued two or three at a time they stalled the waves
            // (bf16 8192 x 8192 x 4096: 858 us, 830 one at a time)
            constexpr int NM = FN * FM - FNG * FM, RS = Q - Q / 4, RP = (ND + RS - 1) / RS;
#pragma unroll
            for (int z = 0; z < Q; ++z) {
                fd.load(z, st, ok, wave);
#pragma unroll
                for (int w = z * RP; w < (z + 1) * RP; ++w) {
                    if (w < FM) f0b[w] = frag_b(nx, 0, w);
                    else if (w < ND) f0a[w - FM] = frag_a(nx, 0, w - FM);
                }
#pragma unroll
                for (int m = FNG * FM + z * NM / Q; m < FNG * FM + (z + 1) * NM / Q; ++m)
                    if (m / FM >= I0 && m / FM < I1)
                        acc[m / FM][m % FM] = CT::step(f1a[m / FM], f1b[m % FM], acc[m / FM][m % FM]);
                __builtin_amdgcn_sched_barrier(0);
            }
            advance();
        };
        if constexpr (!I8) {
            if constexpr (SH::TWO) {
                int kt = 0;
                for (; kt < RF / 2; ++kt) k_step(kt, std::integral_constant<int, 0>{});
                for (; kt < RF; ++kt) k_step(kt, std::integral_constant<int, 1>{});
            } else {
                for (int kt = 0; kt < RF; ++kt) k_step(kt, std::integral_constant<int, 2>{});
            }
            if (RF > 0) {
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FM; ++j) acc[i][j] *= p.scale;
            }
        }
        if constexpr (CT::dt == DT_F32) {
            // (a block's end as a condition in one loop: 77.5 us where this takes 76.5)
            constexpr int BS = SUM_K * CT::es / TL::BKB;   // K steps of a block
            f32x4 done[FN][FM] = {};
            for (int kt = RF; kt < KT;) {
                const int end = KT - kt < BS ? KT : kt + BS;
                for (; kt < end; ++kt) k_step(kt, std::integral_constant<int, 2>{});
#pragma unroll
                for (int i = 0; i < FN; ++i)
#pragma unroll
                    for (int j = 0; j < FM; ++j) {
                        done[i][j] += acc[i][j];
                        acc[i][j] = f32x4{};
                    }
            }
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] += done[i][j];
        } else {
            for (int kt = RF; kt < KT; ++kt) k_step(kt, std::integral_constant<int, 2>{});
        }
        wait_vm<0>();   // the out-of-range loads past the last step still write LDS
    }

    const int g4 = lane >> 4, r = lane & 15;
    if (p.ksplit > 1) {
        // this split's sums; the join applies everything else
        const int64_t MN = p.M * p.N;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int half = SH::TWO ? i / SH::FI : 0;
            const int64_t nb = n0 + wn * SH::WF + (i - half * SH::FI) * 16 + 4 * g4;
            char* part = (char*)p.partial + ((int64_t)blockIdx.y * (SH::TWO ? 2 : 1) + half) * MN * 4;
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const int64_t m = m0 + wm * TL::WM + j * 16 + r;
                if (m >= p.M) continue;
                char* dst = part + (m * p.N + nb) * 4;
                if (nb + 3 < p.N) {
                    ((Any16*)dst)->v = __builtin_bit_cast(i32x4, acc[i][j]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nb + e < p.N) ((int*)dst)[e] = __builtin_bit_cast(i32x4, acc[i][j])[e];
                }
            }
        }
        return;
    }

    // The tile's end works from the accumulators: every output is formed, rounded
    // and written to LDS block by block, so that no second copy of the tile is
    // ever in registers (with one, 77 of them spilled: 8192 x 8192 x 4096 took
    // 910 us, 845 us without).
    __syncthreads();
    if (tid < TL::TN) aux[tid] = bv;
    if (I8) {
        if (tid < TL::TN) aux[TL::TN + tid] = sw;
        if (tid < TL::TM) aux[2 * TL::TN + tid] = sx;
    }
    __syncthreads();
    f32x4 bias4[FN], sw4[I8 ? FN : 1];
    float sxj[I8 ? FM : 1];
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        const int at = (i / SH::FI) * SH::TF + wn * SH::WF + (i % SH::FI) * 16 + 4 * g4;
        bias4[i] = *(const f32x4*)(aux + at);
        if constexpr (I8) sw4[i] = *(const f32x4*)(aux + TL::TN + at);
    }
    if constexpr (I8) {
#pragma unroll
        for (int j = 0; j < FM; ++j) sxj[j] = aux[2 * TL::TN + wm * TL::WM + j * 16 + r];
    }
    // projection `half` of the wave's block (i, j) in fp32
    auto proj = [&](int half, int i, int j) {
        const int ii = half * SH::FI + i;
        f32x4 v = to_f32(acc[ii][j]);
        if constexpr (I8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(v[e] * sw4[ii][e], sxj[j], bias4[ii][e]);
        } else {
            v += bias4[ii];
        }
        return v;
    };
    auto store = [&](auto es, auto val, void* y, int y_dt) {
        store_tile<TL, MODE, decltype(es)::value>(smem, val, y, y_dt, p.M, p.N, n0, m0, wave, lane, wn, wm);
    };
    auto finish = [&](auto es) {
        if constexpr (SH::TWO) {
            with_activation<decltype(es)::value == 4>(p.act, [&](auto act) {
                store(es, [&](int i, int j) {
                    const f32x4 g = proj(0, i, j), v = proj(1, i, j);
                    f32x4 o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = act(g[e]) * v[e];
                    return o;
                }, p.y, p.y_dt);
            });
        } else {
            store(es, [&](int i, int j) { return proj(0, i, j); }, p.y, p.y_dt);
        }
    };
    if constexpr (SH::TWO && !I8) {
        if (p.keep[0] != nullptr) {
            using KES = std::integral_constant<int, CT::es>;
            store(KES{}, [&](int i, int j) { return proj(0, i, j); }, p.keep[0], CT::dt);
            store(KES{}, [&](int i, int j) { return proj(1, i, j); }, p.keep[1], CT::dt);
        }
    }
    if (CT::dt == DT_F32 || p.y_dt == DT_F32) finish(std::integral_constant<int, 4>{});
    else if constexpr (CT::dt != DT_F32) finish(std::integral_constant<int, 2>{});
}

// The K splits' sums joined in split order, then everything the tile's own end
// does.  4 features of a row per thread.
template <class CT, int MODE>
__global__ __launch_bounds__(256) void pair_join_kernel(PairParams p) {
    constexpr bool TWO = MODE == PAIR_PAIR, I8 = CT::dt == DT_I8;
    const int64_t per_row = (p.N + 3) / 4, MN = p.M * p.N;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.M * per_row) return;
    const int64_t m = i / per_row, n = (i - m * per_row) * 4;
    const int cnt = (int)(p.N - n < 4 ? p.N - n : 4);
    f32x4 pr[TWO ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (TWO ? 2 : 1); ++h) {
        Acc<CT> sum{};
        for (int k = 0; k < p.ksplit; ++k) {
            const char* src = (const char*)p.partial + (((int64_t)k * (TWO ? 2 : 1) + h) * MN + m * p.N + n) * 4;
            i32x4 raw = i32x4{0, 0, 0, 0};
            if (cnt == 4) {
                raw = ((const Any16*)src)->v;
            } else {
                for (int e = 0; e < cnt; ++e) raw[e] = ((const int*)src)[e];
            }
            sum += __builtin_bit_cast(Acc<CT>, raw);
        }
        f32x4 v = to_f32(sum);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = e < cnt;
            const float b = p.bias[h] != nullptr && in ? load_as_f32(p.bias[h], p.bias_dt, n + e) : 0.f;
            if constexpr (I8) v[e] = __builtin_fmaf(v[e] * (in ? p.sw[h][n + e] : 0.f), p.sx[m], b);
            else v[e] += b;
        }
        pr[h] = v;
    }
    auto put = [&](void* y, int dt, const f32x4& v) {
        const int64_t at = m * p.N + n;
        for (int e = 0; e < cnt; ++e) {
            if (dt == DT_F32) ((float*)y)[at + e] = v[e];
            else ((uint16_t*)y)[at + e] = dt == DT_F16 ? f32_to_f16(v[e]) : f32_to_bf16(v[e]);
        }
    };
    if constexpr (TWO) {
        if (!I8 && p.keep[0] != nullptr) {
            put(p.keep[0], CT::dt, pr[0]);
            put(p.keep[1], CT::dt, pr[1]);
        }
        with_activation<true>(p.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[0][e] = act(pr[0][e]) * pr[1][e];
        });
    }
    put(p.y, p.y_dt, pr[0]);
}

// ---- few token rows: one workgroup per 16 FB features ----------------------------
// M <= 32 with all of K in one workgroup: wave w of the NW takes the w-th share
// of the 64-byte K steps, its fragments read straight from global memory D
// steps ahead (every weight byte is used once, so nothing is staged); wave 0
// takes the folds first.  The waves' sums meet in LDS in wave order.  Bound by
// the weights' bytes.
template <class CT, int MODE, int MT, int FB, int D, int NW>
__global__ __launch_bounds__(64 * NW) void pair_skinny_kernel(PairParams p) {
    constexpr bool TWO = MODE == PAIR_PAIR, I8 = CT::dt == DT_I8;
    static_assert(!TWO || FB == 1, "16 features of both matrices");
    constexpr int H = TWO ? 2 : FB, SEGS = MODE == PAIR_SEQ ? 2 : 1;   // 16-row blocks of weights; products
    __shared__ __attribute__((aligned(16))) Acc<CT> red[NW][H][MT][64];
    const int tid = threadIdx.x, lane = tid & 63, g4 = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * FB);
    const uint32_t kb = (uint32_t)(p.K * CT::es), lo = (uint32_t)g4 * 16;
    const uint32_t nrows = (uint32_t)(p.N - n0 < 16 * FB ? p.N - n0 : 16 * FB);   // (of each matrix)
    Acc<CT> acc[H][MT];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[h][t] = Acc<CT>{};

    if constexpr (!I8) {
        if (wave == 0 && p.rf > 0) {
            const uint32_t fb = (uint32_t)(p.rf * CT::es), ld = (uint32_t)(p.ldf * CT::es);
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const auto ru = make_rsrc_uniform((const char*)p.af[f] + n0 * fb, nrows * fb);
                const auto rh = make_rsrc_uniform(p.bf[f], (uint32_t)(p.M - 1) * ld + fb);
                for (uint32_t k = 0; k < fb; k += 64) {
                    const bool in = k + lo < fb;
                    i32x4 hb[MT];
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const bool on = in && 16 * t + r < p.M;
                        hb[t] = buf_load16(rh, on ? (uint32_t)(16 * t + r) * ld + k + lo : OOB);
                    }
#pragma unroll
                    for (int h = TWO ? f : 0; h < (TWO ? f + 1 : H); ++h) {
                        const uint32_t row = (uint32_t)(TWO ? r : 16 * h + r);
                        const i32x4 ua = buf_load16(ru, in ? row * fb + k + lo : OOB);
#pragma unroll
                        for (int t = 0; t < MT; ++t) acc[h][t] = CT::step(ua, hb[t], acc[h][t]);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[h][t] *= p.scale;
        }
    }

    // ring slot u holds step s0 + u (mod D); the run is padded to a multiple of
    // D with steps that read zeros, so the loop body has no exit in it and the
    // ring stays in flight across iterations
    const int steps = (int)((kb + 63) / 64);
    const int s0 = steps * wave / NW, s1 = steps * (wave + 1) / NW;
    const int se = s0 + ((s1 - s0 + D - 1) / D) * D;
    constexpr bool BLOCKS = CT::dt == DT_F32;
    constexpr int BS = SUM_K * CT::es / 64;   // steps of a block
    static_assert((BS & (BS - 1)) == 0 && BS % D == 0, "steps of a block");
    Acc<CT> done[BLOCKS ? H : 1][BLOCKS ? MT : 1] = {};
#pragma unroll
    for (int sg = 0; sg < SEGS; ++sg) {
        const auto rx = make_rsrc_uniform(p.b[sg], (uint32_t)p.M * kb);
        const auto rw0 = make_rsrc_uniform((const char*)p.a[sg] + n0 * kb, nrows * kb);
        const auto rw1 = make_rsrc_uniform((const char*)p.a[TWO ? 1 : sg] + n0 * kb, nrows * kb);
        i32x4 wa[D][H], xa[D][MT];
        auto load = [&](int u, int s) {
            const uint32_t k = (uint32_t)s * 64 + lo;
            const bool in = s < s1 && k < kb;
#pragma unroll
            for (int h = 0; h < H; ++h)
                wa[u][h] = buf_load16(TWO && h ? rw1 : rw0, in ? (uint32_t)(TWO ? r : 16 * h + r) * kb + k : OOB);
#pragma unroll
            for (int t = 0; t < MT; ++t) xa[u][t] = buf_load16(rx, in ? (uint32_t)(16 * t + r) * kb + k : OOB);
        };
#pragma unroll
        for (int u = 0; u < D; ++u) load(u, s0 + u);
        for (int sb = s0; sb < se; sb += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int t = 0; t < MT; ++t) acc[h][t] = CT::step(wa[u][h], xa[u][t], acc[h][t]);
                load(u, sb + u + D);
            }
            if (BLOCKS && ((sb - s0) & (BS - 1)) == BS - D) {
#pragma unroll
                for (int h = 0; h < (BLOCKS ? H : 0); ++h)
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        done[h][t] += acc[h][t];
                        acc[h][t] = Acc<CT>{};
                    }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < (BLOCKS ? H : 0); ++h)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[h][t] += done[h][t];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int t = 0; t < MT; ++t) red[wave][h][t][lane] = acc[h][t];
    __syncthreads();
    static_assert(MT * (TWO ? 1 : H) <= NW, "a wave per output block");
    if (wave >= MT * (TWO ? 1 : H)) return;
    // wave t (ONE, SEQ: + MT times the block of features) ends rows m = 16 t + r,
    // features nb .. nb + 3
    const int mt = wave % MT, fb0 = TWO ? 0 : wave / MT;
    const int64_t m = 16 * mt + r, nb = n0 + 16 * fb0 + 4 * g4;
    if (m >= p.M) return;
    f32x4 pr[TWO ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (TWO ? 2 : 1); ++h) {
        Acc<CT> sum = red[0][fb0 + h][mt][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) sum += red[w][fb0 + h][mt][lane];
        f32x4 v = to_f32(sum);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = nb + e < p.N;
            const float b = p.bias[h] != nullptr && in ? load_as_f32(p.bias[h], p.bias_dt, nb + e) : 0.f;
            if constexpr (I8) v[e] = __builtin_fmaf(v[e] * (in ? p.sw[h][nb + e] : 0.f), p.sx[m], b);
            else v[e] += b;
        }
        pr[h] = v;
    }
    auto put = [&](void* y, int dt, const f32x4& v) {
        const int64_t at = m * p.N + nb;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (nb + e >= p.N) continue;
            if (dt == DT_F32) ((float*)y)[at + e] = v[e];
            else ((uint16_t*)y)[at + e] = dt == DT_F16 ? f32_to_f16(v[e]) : f32_to_bf16(v[e]);
        }
    };
    if constexpr (TWO) {
        if (!I8 && p.keep[0] != nullptr) {
            put(p.keep[0], CT::dt, pr[0]);
            put(p.keep[1], CT::dt, pr[1]);
        }
        with_activation<true>(p.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[0][e] = act(pr[0][e]) * pr[1][e];
        });
    }
    put(p.y, p.y_dt, pr[0]);
}

// ---- launchers shared by the instances' files -------------------------------------

using PairL = Tile<256, 256, 128, 64, 2, 128>;   // 8 waves, 128 KiB of stages
using PairM = Tile<128, 128, 64, 32, 4, 128>;    // 8 waves, 128 KiB
using PairF = Tile<96, 128, 96, 32, 4, 128>;     // 4 waves, 112 KiB: fp32 only
using PairS = Tile<64, 64, 32, 32, 4, 128>;      // 4 waves, 64 KiB

template <class CT, class TL, int MODE>
hipError_t run_pair(const PairParams& p, hipStream_t s) {
    using SH = PairShape<TL, MODE>;
    const int64_t tiles_n = (p.N + SH::TF - 1) / SH::TF, tiles_m = (p.M + TL::TM - 1) / TL::TM;
    if (tiles_n * tiles_m >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    const int ks = p.ksplit > 1 ? p.ksplit : 1;
    hipLaunchKernelGGL((pair_kernel<CT, TL, MODE>), dim3((unsigned)(tiles_n * tiles_m), ks), dim3(TL::NT), 0, s, p,
                       (int)tiles_n, (int)tiles_m, 4);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || ks == 1) return e;
    const int64_t groups = p.M * ((p.N + 3) / 4);
    hipLaunchKernelGGL((pair_join_kernel<CT, MODE>), dim3((unsigned)((groups + 255) / 256)), dim3(256), 0, s, p);
    return hipGetLastError();
}

// The few-row kernel's x rows are read by every workgroup, from L2: 32 features
// a workgroup halve that where they still leave one per CU
bool pair_wide(int64_t N);
// 32-bit offsets of the few-row kernel
inline bool pair_skinny(int64_t M, int64_t K, int es) {
    return M >= 1 && M <= 32 && K > 0 && 32 * K * es < ((int64_t)1 << 31);
}

template <class CT, int MODE, int FB>
hipError_t run_pair_skinny(const PairParams& p, hipStream_t s) {
    const dim3 g((unsigned)((p.N + 16 * FB - 1) / (16 * FB)));
    // 4 waves, 4 steps ahead, 2 where two blocks of rows double the registers: int8
    // 16 x 8192 x 8192 16.4 us (8 ahead 18.2, 12 19.6, 2 17.6; 8 waves 20.8), 32 x 8192 x
    // 8192 19.6 (4 ahead 21.1, 6 22.7)
    if (p.M <= 16) hipLaunchKernelGGL((pair_skinny_kernel<CT, MODE, 1, FB, 4, 4>), g, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((pair_skinny_kernel<CT, MODE, 2, FB, 2, 4>), g, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <class CT, int MODE>
hipError_t run_pair_ct(const PairParams& p, hipStream_t s) {
    if (p.ksplit <= 1 && pair_skinny(p.M, p.K, CT::es)) {
        if constexpr (MODE != PAIR_PAIR) {
            if (pair_wide(p.N)) return run_pair_skinny<CT, MODE, 2>(p, s);
        }
        return run_pair_skinny<CT, MODE, 1>(p, s);
    }
    const PairPlan pl = pair_plan(MODE, CT::dt, p.M, p.N, p.K);
    if (p.ksplit > 1 && p.partial == nullptr) return hipErrorInvalidValue;
    if constexpr (CT::dt != DT_F32) {
        if (pl.tile_m == 256) return run_pair<CT, PairL, MODE>(p, s);
    }
    if constexpr (CT::dt == DT_F32) {
        if (pl.tile_m == 128 && pl.tile_n == PairShape<PairF, MODE>::TF) return run_pair<CT, PairF, MODE>(p, s);
    }
    if (pl.tile_m == 128) return run_pair<CT, PairM, MODE>(p, s);
    return run_pair<CT, PairS, MODE>(p, s);
}

}  // namespace lyc
