// ortho.h -- host-side launcher of the Newton-Schulz orthogonalization
// (internal to the library; the public surface is include/lyc.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lyc {

constexpr int ORTHO_MAX_STEPS = 32;

struct OrthoParams {
    const void* g;   // [R][C], row-major
    int dt;          // dtype of g and out
    void* out;       // [R][C]
    int64_t R, C;
    int steps;
    double a, b, c;  // X <- a X + (b A + c A^2) X, A = X X^T over the short side
    double eps;      // X0 = g / (|g|_F + eps)
    char* ws;        // ortho_workspace(R, C, dt) bytes, 256-byte aligned
};
size_t ortho_workspace(int64_t R, int64_t C, int dt);
// a dense update's product (0: A, 1: P, 2: P X); tile 0 where there is none
struct OrthoPlan {
    int tile_n, tile_m, ksplit, halved;
};
OrthoPlan ortho_plan(int64_t R, int64_t C, int dt, int product);
hipError_t launch_ortho(const OrthoParams& p, hipStream_t s);

}  // namespace lyc
