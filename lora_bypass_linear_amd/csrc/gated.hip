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

PairPlan pair_plan(int mode, int c_dt, int64_t M, int64_t N, int64_t K) {
    const int es = c_dt == DT_F32 ? 4 : c_dt == DT_I8 ? 1 : 2;
    const int two = mode == PAIR_PAIR ? 2 : 1;
    if (M <= 0 || N <= 0) return PairPlan{0, 0, 1};
    if (pair_skinny(M, K, es)) return PairPlan{16, M <= 16 ? 16 : 32, 1};
    struct C {
        int t, per_cu;
        double fixed, step;
    };
    const C cands[3] = {{256, 1, 8.0, 1.15}, {128, 1, 6.0, 0.42}, {64, 2, 5.0, 0.45}};
    const double cus = (double)device_rates().cus;
    const int64_t steps1 = (K * es + 127) / 128;
    const double seg = mode == PAIR_SEQ ? 2.0 : 1.0;
    PairPlan best{64 / two, 64, 1};
    double best_t = 1e300;
    for (const C& c : cands) {
        if (c_dt == DT_F32 && c.t == 256) continue;
        const double f32 = c_dt == DT_F32 ? 8.0 : 1.0;
        const int tf = c.t / two;
        const double tiles = (double)((N + tf - 1) / tf) * (double)((M + c.t - 1) / c.t);
        for (int ks = 1; ks <= 8; ks *= 2) {
            const double part = (double)M * N * 4.0 * two * ks;
            if (ks > 1 && (ks > steps1 / 2 || part > 64.0 * 1024 * 1024)) continue;
            const double st = (double)((steps1 + ks - 1) / ks) * seg;
            double t = std::ceil(tiles * ks / (cus * c.per_cu)) * (c.fixed + st * c.step * f32);
            if (ks > 1) t += 3.0 + part * (1.0 + 1.0 / ks) / 2.5e6;
            if (t < best_t) {
                best_t = t;
                best = PairPlan{tf, c.t, ks};
            }
        }
    }
    return best;
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
