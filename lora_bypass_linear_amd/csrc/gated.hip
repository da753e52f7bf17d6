// gated.hip -- the gated feed-forward block's forward on gfx950 MFMA,
//
//   y = round_out( act(g) * v ),  g, v = x.W^T + scale * h_r.up^T + b  of gate and value
//
// (pair_tile.h, PAIR), and the plan that every product of that file runs with.
#include <algorithm>
#include <cmath>

#include "kernels.h"
#include "pair_tile.h"

namespace lyc {

hipError_t launch_gated(int c_dt, const PairParams& p, hipStream_t s) {
    if (c_dt == DT_F16) return run_pair_ct<CF16, PAIR_PAIR>(p, s);
    if (c_dt == DT_BF16) return run_pair_ct<CBF16, PAIR_PAIR>(p, s);
    return run_pair_ct<CF32, PAIR_PAIR>(p, s);
}

bool pair_wide(int64_t N) { return N >= 32 * device_rates().cus; }

// Tile and K split by modelled time, us: rounds of workgroups over the CUs (two
// 64 x 64 ones share one), each a fixed part and its K steps of 128 bytes a row,
// whose time grows with the share of the device that is busy; plus a split's
// sums out and in again.  Measured steps, on an empty and on a full device
// (rows x A rows of a tile; the byte widths of the operands do not matter):
//             8 and 16 bits          fp32
//   256 x 256    0.8, 1.42  fixed 12.5     --
//   128 x 128    0.37, 0.53       5      2.0, 2.2
//   128 x 96         --                  1.5, 1.8     5
//   64 x 64      0.22, 0.37       5      0.5, 1.06
// Whole calls, the pick and what it is held against: int8 product 777 x 4104 x
// 4112 128 x 128 24.4, 64 x 64 39.5, 256 x 256 in two splits 45.5; 512 x 512 x 8192
// 64 x 64 in 4 splits 13.7, in one 21.5; bf16 block 777 x 4096 x 4096 128 x 128
// 67.2, 256 x 256 80.3; 256 x 4096 x 4096 64 x 64 28.7, 128 x 128 33.0; fp32 block 200 x
// 512 x 4096 64 x 64 in 4 splits 32.2, in one 83.7; 517 x 2056 x 1032 128 x 96 75.9, 64 x
// 64 79.4.
PairPlan pair_plan(int mode, int c_dt, int64_t M, int64_t N, int64_t K) {
    const int es = c_dt == DT_F32 ? 4 : c_dt == DT_I8 ? 1 : 2;
    const int two = mode == PAIR_PAIR ? 2 : 1;
    if (M <= 0 || N <= 0) return PairPlan{0, 0, 1};
    if (pair_skinny(M, K, es)) return PairPlan{two == 1 && pair_wide(N) ? 32 : 16, M <= 16 ? 16 : 32, 1};
    struct C {
        int a, t, per_cu;   // rows of A and of B, workgroups a CU holds
        double fixed, empty, full;
    };
    const C cands[2][3] = {{{256, 256, 1, 12.5, 0.8, 1.42}, {128, 128, 1, 5.0, 0.37, 0.53}, {64, 64, 2, 5.0, 0.22, 0.37}},
                           {{128, 128, 1, 5.0, 2.0, 2.2}, {96, 128, 1, 5.0, 1.5, 1.8}, {64, 64, 2, 5.0, 0.5, 1.06}}};
    const double cus = (double)device_rates().cus;
    const int64_t steps1 = (K * es + 127) / 128;
    const double segs = mode == PAIR_SEQ ? 2.0 : 1.0;
    PairPlan best{64 / two, 64, 1};
    double best_t = 1e300;
    for (const C& c : cands[c_dt == DT_F32 ? 1 : 0]) {
        const int tf = c.a / two;
        const double tiles = (double)((N + tf - 1) / tf) * (double)((M + c.t - 1) / c.t);
        for (int ks = 1; ks <= 8; ks *= 2) {
            const double part = (double)M * (double)N * 4.0 * two * ks;
            if (ks > 1 && (ks > steps1 / 2 || part > 64.0 * 1024 * 1024)) continue;
            const double steps = (double)((steps1 + ks - 1) / ks) * segs;
            const double slots = cus * c.per_cu, rounds = std::ceil(tiles * ks / slots);
            const double busy = tiles * ks / (rounds * slots);
            double t = rounds * (c.fixed + steps * (c.empty + (c.full - c.empty) * busy));
            if (ks > 1) t += 2.5 + 2.0 * part / 3.0e6;
            if (t < best_t) {
                best_t = t;
                best = PairPlan{tf, c.t, ks};
            }
        }
    }
    return best;
}

bool pair_fits(int mode, int c_dt, int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0) return true;
    const PairPlan p = pair_plan(mode, c_dt, M, N, K);
    const int64_t wgs = ((N + p.tile_n - 1) / p.tile_n) * ((M + p.tile_m - 1) / p.tile_m);
    return wgs * (p.tile_m >= 128 ? 512 : 256) < ((int64_t)1 << 32);
}

hipError_t launch_gated(int c_dt, const PairParams& p, hipStream_t s);
hipError_t launch_seq(int c_dt, const PairParams& p, hipStream_t s);
hipError_t launch_int8(int mode, const PairParams& p, hipStream_t s);

hipError_t launch_pair(int mode, int c_dt, const PairParams& p, hipStream_t s) {
    if (p.M <= 0 || p.N <= 0) return hipSuccess;
    if (c_dt == DT_I8) return mode == PAIR_SEQ ? hipErrorInvalidValue : launch_int8(mode, p, s);
    if (mode == PAIR_PAIR) return launch_gated(c_dt, p, s);
    return mode == PAIR_SEQ ? launch_seq(c_dt, p, s) : hipErrorInvalidValue;
}

}  // namespace lyc
