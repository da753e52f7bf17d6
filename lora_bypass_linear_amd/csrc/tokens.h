// tokens.h -- host-side launcher of the gated backward's contractions over the
// tokens (internal to the library; the public surface is include/lyc.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lyc {

// S[c][j] = sum_m wide[m][c] rank[m][j], c < C, j < r, both in the 16-bit compute
// dtype with 16-byte aligned rows; out = round_out(post * S), as [r][C] (by_rank)
// or [C][r]
struct TokenJob {
    const void* wide;   // [M][C], C a multiple of 8
    int64_t C;
    const void* rank;   // [M][ldr], r columns used (more are read, never past row M)
    int64_t ldr, r;
    void* out;
    int out_dt;
    int by_rank;
    float post;
};
// bytes of a split's sums for d_down (dd) and d_up (du) of both projections
size_t tokens_partial(int64_t M, int64_t K, int64_t N, int64_t r, bool dd, bool du);
// up to 4 jobs of one r in one launch (plus one that joins the splits)
hipError_t launch_tokens(int c_dt, const TokenJob* jobs, int n, int64_t M, float* partial, hipStream_t s);

}  // namespace lyc
