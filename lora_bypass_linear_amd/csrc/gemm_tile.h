// gemm_tile.h -- what the tiled MFMA products share: the output tile's shape,
// the workgroup -> tile mapping, the direct-to-LDS loader of K-contiguous
// operands and the whole-row epilogue.
#pragma once

#include "kernels.h"
#include "lyc_device.h"

namespace lyc {

// TN x TM output tile, WN x WM per wave (multiples of 16), NS pipeline stages
// of one K step each.  A K step is BKB bytes of every row (64: 32 16-bit
// values; 128: 64), made of SUB = BKB/64 MFMA substeps of 64 bytes.
template <int TN_, int TM_, int WN_, int WM_, int NS_, int BKB_>
struct Tile {
    static constexpr int TN = TN_, TM = TM_, WN = WN_, WM = WM_, NS = NS_, BKB = BKB_;
    static constexpr int WAVES_N = TN / WN, WAVES_M = TM / WM;
    static constexpr int NW = WAVES_N * WAVES_M, NT = NW * 64;
    static constexpr int FN = WN / 16, FM = WM / 16;
    static constexpr int SUB = BKB / 64;                        // MFMA substeps per K step
    static constexpr int CH = BKB / 16;                         // 16-byte chunks per row
    static constexpr int RPB = 64 / CH;                         // rows per 1 KiB wave load
    static constexpr int NBLK = (TN + TM) / RPB;                // wave loads per step
    static constexpr int Q = NBLK / NW;                         // loads per wave per step
    static constexpr int STAGE = (TN + TM) * BKB;               // LDS bytes per stage
    static_assert(BKB == 64 || BKB == 128, "K step");
    static_assert(TN % WN == 0 && TM % WM == 0 && WN % 16 == 0 && WM % 16 == 0, "tile shape");
    static_assert(NBLK % NW == 0 && Q >= 1, "loader split");
    static_assert(NS >= 2 && NS * STAGE <= 160 * 1024, "LDS");
    static_assert((NS - 1) * Q < 64, "vmcnt range");
};

// Workgroup id -> output tile.  Workgroups are dispatched round-robin over the
// 8 XCDs (id % 8), each with its own L2: give every XCD a contiguous range of
// logical tiles, and walk that range in groups of `group_m` m-tiles so the
// tiles resident on one XCD share W and x rows in its L2.
__device__ __forceinline__ void tile_coords(int bid, int nblk, int tiles_n, int tiles_m, int group_m, int& tn,
                                            int& tm) {
    const int per = nblk >> 3, rem = nblk & 7;
    const int xcd = bid & 7, loc = bid >> 3;
    const int l = xcd * per + (xcd < rem ? xcd : rem) + loc;
    const int in_group = group_m * tiles_n;
    const int g = l / in_group;
    const int first_m = g * group_m;
    const int gsz = (tiles_m - first_m) < group_m ? (tiles_m - first_m) : group_m;
    const int r = l - g * in_group;
    tm = first_m + r % gsz;
    tn = r / gsz;
}

// LDS rows hold BKB bytes (CH chunks of 16).  Chunk kc of row r sits at slot
// kc ^ swz(r), swz(r) = (r / (128 / BKB)) mod CH, so the 16-byte fragment
// reads of 8 consecutive rows (one or two rows per 128 bytes) hit 8 different
// bank groups.
template <class TL>
__device__ __forceinline__ int swz(int row) {
    return TL::BKB == 128 ? (row & 7) : ((row >> 1) & 3);
}
template <class TL>
__device__ __forceinline__ int lds_at(int row, int kc) {
    return row * TL::BKB + ((kc ^ swz<TL>(row)) << 4);
}

// Global -> LDS without registers: one buffer_load_dwordx4 ... lds per wave
// fills 1 KiB of LDS = RPB rows x BKB bytes of a K step.  The LDS side of such
// a load is fixed (lane l writes bytes 16l .. 16l+15 of the KiB), so each lane
// fetches the global chunk that belongs in that slot of the swizzled layout:
// row RPB blk + l / CH, logical chunk (l mod CH) ^ swz(that row).  The blocks of
// the A (W-side) and B (x-side) tiles are numbered together and dealt to the
// waves round-robin.
template <class TL>
struct Loader {
    // The blocks of the A (W-side) and B (x-side) tiles are dealt round-robin,
    // so a wave's load q covers A block wave + q NW (q < QA) or B block
    // wave + (q - QA) NW: its lane offset is the lane's offset in the wave's
    // first block of that side plus a uniform stride.
    static constexpr int QA = TL::TN / TL::RPB / TL::NW, QB = TL::TM / TL::RPB / TL::NW;
    static_assert(QA * TL::RPB * TL::NW == TL::TN && QB * TL::RPB * TL::NW == TL::TM, "loader split");
    uint32_t va, vb;          // lane offsets in the first A / B block, k step 0
    uint32_t sa, sb;          // byte stride between a wave's consecutive blocks (uniform)
    __device__ __forceinline__ static uint32_t chunk16(int lane) {
        return (uint32_t)((lane % TL::CH) ^ swz<TL>(lane / TL::CH)) << 4;
    }
    __device__ __forceinline__ void init(uint32_t a_bytes, uint32_t b_bytes, int wave, int lane) {
        const uint32_t row = (uint32_t)(wave * TL::RPB + lane / TL::CH);
        va = row * a_bytes + chunk16(lane);
        vb = row * b_bytes + chunk16(lane);
        sa = (uint32_t)(TL::NW * TL::RPB) * a_bytes;
        sb = (uint32_t)(TL::NW * TL::RPB) * b_bytes;
    }
    // loads of one K step (kb0 = its first byte within a row) into an LDS stage;
    // rows past a tile's valid rows read zeros through the buffer range check
    // (the row offset is in the range-checked vector offset), and in the last,
    // ragged step the chunks past the row end are sent out of range too
    template <bool DO_A = true, bool DO_B = true>
    __device__ __forceinline__ void issue(char* stage, __amdgpu_buffer_rsrc_t ra, __amdgpu_buffer_rsrc_t rb,
                                          uint32_t row_bytes, uint32_t kb0, int wave, int lane) const {
        const bool ok = kb0 + TL::BKB <= row_bytes || kb0 + chunk16(lane) < row_bytes;
#pragma unroll
        for (int q = 0; q < (DO_A ? QA : 0); ++q) {
            const uint32_t v = ok ? va + (uint32_t)q * sa : OOB;
            auto* dst = (__attribute__((address_space(3))) void*)(stage + (wave + q * TL::NW) * 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, dst, 16, v, (int)kb0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < (DO_B ? QB : 0); ++q) {
            const uint32_t v = ok ? vb + (uint32_t)q * sb : OOB;
            auto* dst = (__attribute__((address_space(3))) void*)(stage + (wave + (QA + q) * TL::NW) * 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, dst, 16, v, (int)kb0, 0, 0);
        }
    }
};

// The output tile through LDS, so that every store writes whole rows of it.
// A lane's MFMA results are 4 consecutive n of one token row m for each 16x16
// block, so a store straight from them covers 16 rows x 8-16 bytes: at the
// bf16 16384 x 8192 x 8192 size those partial-line stores took ~9 us at the
// end of each tile.  Here the waves write their blocks (scaled, biased,
// rounded to y's dtype) into the free pipeline stages as rows of the tile
// (16-byte chunk c of row r at slot c ^ (r & 7)), and then store 16-byte
// chunks in row order: a wave's store covers 1 KiB of consecutive rows.  A
// tile larger than the stages (fp32 output of the 256-row tiles) goes in two
// passes of half its rows.  Needs N * ES a multiple of 16 and y 16-byte
// aligned (a chunk is then all inside y's row or all past its end).
template <class TL, int ES, bool GAIN>
__device__ __forceinline__ void epilogue_rows(const GemmParams& p, char* smem, const f32x4 (&acc)[TL::FN][TL::FM],
                                              const float* biasv, const float* gainv, int64_t n0, int64_t m0,
                                              int wave, int lane, int wn, int wm) {
    constexpr int RB = TL::TN * ES, CHR = RB / 16;   // bytes and 16-byte chunks of a tile row
    constexpr int CAP = TL::NS * TL::STAGE;
    constexpr int TMP = TL::TM * RB <= CAP ? TL::TM : TL::TM / 2;   // rows per pass
    constexpr int PASSES = TL::TM / TMP, IT = TMP * CHR / (TL::NW * 64);
    static_assert(TMP * RB <= CAP && TL::TM % TMP == 0 && TMP % TL::WM == 0 && CHR % 8 == 0, "staged rows");
    static_assert(IT * TL::NW * 64 == TMP * CHR, "whole wave stores");
    const int64_t yrow = p.N * ES;
    // (the barriers fence the scheduler, and the stores go four chunks at a
    // time: with two passes the second pass's writers still hold their
    // accumulators during the first pass's stores, and a deeper batch, or
    // outputs computed ahead of a barrier, made the registers spill)
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
        __syncthreads();   // the stages (then the previous pass's rows) are free
        __builtin_amdgcn_sched_barrier(0);
        if ((wm * TL::WM) / TMP == ps) {
#pragma unroll
            for (int i = 0; i < TL::FN; ++i) {
                const int nl = wn * TL::WN + i * 16 + 4 * (lane >> 4);
                const float* bias = biasv + 4 * i;
                const float* gain = gainv + (GAIN ? 4 * i : 0);
#pragma unroll
                for (int j = 0; j < TL::FM; ++j) {
                    const int r = wm * TL::WM + j * 16 + (lane & 15) - ps * TMP;
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * (GAIN ? gain[e] : p.post) + bias[e];
                    const int cb = nl * ES;   // byte column
                    char* dst = smem + r * RB + ((((cb >> 4) ^ (r & 7)) << 4) | (cb & 15));
                    if constexpr (ES == 4) {
                        *(f32x4*)dst = f32x4{v[0], v[1], v[2], v[3]};
                    } else {
                        const uint32_t lo = p.y_dt == DT_F16 ? pack_f16x2(v[0], v[1]) : pack_bf16x2(v[0], v[1]);
                        const uint32_t hi = p.y_dt == DT_F16 ? pack_f16x2(v[2], v[3]) : pack_bf16x2(v[2], v[3]);
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
            const i32x4 d = *(const i32x4*)(smem + r * RB + ((c ^ (r & 7)) << 4));
            const int64_t m = m0 + ps * TMP + r, n = n0 + c * (16 / ES);
            if (m < p.M && n < p.N) *(i32x4*)((char*)p.y + m * yrow + n * ES) = d;
        }
    }
}

}  // namespace lyc
