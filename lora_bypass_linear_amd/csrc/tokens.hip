// tokens.hip -- the gated block's four factor gradients, contracted over the
// tokens, in one launch:
//
//   d_down_p[j][k] = sum_m gh_p[m][j] x[m][k]          wide = x,   rank side = gh_p
//   d_up_p[n][j]   = scale * sum_m d_p[m][n] h_p[m][j]   wide = d_p, rank side = h_p
//
// Both sides are stored with the tokens as rows, so a step of 64 tokens is staged
// in LDS as it lies in memory and turned into MFMA fragments by the transposing
// LDS reads.  One workgroup takes 128 columns of the wide side and the whole rank
// side (padded to 64, 128 or 256), so that the wide matrices stream through once
// per product; the rank side, re-read by every workgroup, comes from L2.  Few
// columns leave CUs idle, so the tokens are split too; the splits' fp32 sums are
// added in split order by a second kernel.  Bound by the wide sides' bytes: bf16
// 8192 tokens, 4096 and 8192 columns, rank 64: 92 us for all four (4.4 TB/s) and 10
// for the join; as four GEMM launches with their reductions 135 us.
#include "kernels.h"
#include "lyc_device.h"
#include "tokens.h"

namespace lyc {

constexpr int TK_C = 128, TK_T = 64, TK_NS = 3;   // wide columns, tokens a step, stages

struct TokenLaunch {
    TokenJob job[4];
    int end[4];       // column tiles up to and with each job
    int64_t at[4];    // its first element in a split's sums
    int64_t M, total;
    int jobs, splits;
    float* partial;
};

// a step's rows of one side: ROWS columns from base, 1 KiB a wave load
template <int ROWS>
struct TokenSide {
    static constexpr int CPR = ROWS / 8, KRB = 64 / CPR, LOADS = TK_T / KRB / 4;
    static_assert(LOADS * KRB * 4 == TK_T, "4 waves");
    const char* base;
    uint32_t ld, range;
    __device__ __forceinline__ void init(const void* p, int64_t col0, int64_t ld_, int64_t M) {
        base = (const char*)p + col0 * 2;
        ld = (uint32_t)ld_ * 2;
        range = (uint32_t)(M * ld_ * 2 - col0 * 2);
    }
    __device__ __forceinline__ void issue(char* lds, int64_t step, bool on, int wave, int lane) const {
        const auto r = make_rsrc(base, on ? range : 0u);
#pragma unroll
        for (int q = 0; q < LOADS; ++q) {
            const int row = (wave + q * 4) * KRB + lane / CPR;
            const uint32_t off = (uint32_t)(step * TK_T + row) * ld + (uint32_t)((lane % CPR) ^ tswz<CPR>(row)) * 16;
            auto* dst = (__attribute__((address_space(3))) void*)(lds + (wave + q * 4) * 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, off, 0, 0, 0);
        }
    }
};

template <class CT, int RT>
__global__ __launch_bounds__(256) void tokens_kernel(TokenLaunch p) {
    constexpr int WIDE = TK_T * TK_C * 2, STAGE = WIDE + TK_T * RT * 2, JB = RT / 16;
    using W = TokenSide<TK_C>;
    using R = TokenSide<RT>;
    constexpr int Q = W::LOADS + R::LOADS;
    __shared__ __attribute__((aligned(16))) char smem[TK_NS * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int k = 0;
    while ((int)blockIdx.x >= p.end[k]) ++k;
    const TokenJob job = p.job[k];
    const int64_t c0 = (int64_t)((int)blockIdx.x - (k > 0 ? p.end[k - 1] : 0)) * TK_C;
    W sw;
    R sr;
    sw.init(job.wide, c0, job.C, p.M);
    sr.init(job.rank, 0, job.ldr, p.M);
    const int64_t steps = (p.M + TK_T - 1) / TK_T;
    const int64_t s0 = steps * blockIdx.y / p.splits, s1 = steps * (blockIdx.y + 1) / p.splits;
    f32x4 acc[2][JB];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (steps past the last are out of range: every step issues the same loads)
    auto issue = [&](int64_t s) {
        char* st = smem + (int)((s - s0) % TK_NS) * STAGE;
        sw.issue(st, s, s < s1, wave, lane);
        sr.issue(st + WIDE, s, s < s1, wave, lane);
    };
#pragma unroll
    for (int s = 0; s < TK_NS - 1; ++s) issue(s0 + s);
    for (int64_t s = s0; s < s1; ++s) {
        wait_vm<(TK_NS - 2) * Q>();
        lds_barrier();   // step s has landed for every wave, and step s - 1 has been read
        issue(s + TK_NS - 1);
        const char* st = smem + (int)((s - s0) % TK_NS) * STAGE;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            i32x4 a[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) a[i] = frag_t<TK_C>(st, sub * 32, wave * 32 + i * 16, lane);
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                const i32x4 b = frag_t<RT>(st + WIDE, sub * 32, j * 16, lane);
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[i][j] = CT::step(a[i], b, acc[i][j]);
            }
        }
    }
    wait_vm<0>();   // the out-of-range loads past the last step still write LDS
    // lane: columns c0 + 32 wave + 16 i + 4 (lane / 16) .. + 3 of rank column 16 j + lane % 16
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t c = c0 + wave * 32 + i * 16 + 4 * (lane >> 4);
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int64_t rj = j * 16 + (lane & 15);
            if (rj >= job.r || c >= job.C) continue;   // (C is a multiple of 8: four columns are in or out)
            const f32x4 v = acc[i][j];
            if (p.splits > 1) {
                float* dst = p.partial + (int64_t)blockIdx.y * p.total + p.at[k];
                if (job.by_rank) {
                    *(f32x4*)(dst + rj * job.C + c) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[(c + e) * job.r + rj] = v[e];
                }
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t at = job.by_rank ? rj * job.C + c + e : (c + e) * job.r + rj;
                const float x = v[e] * job.post;
                if (job.out_dt == DT_F32) ((float*)job.out)[at] = x;
                else ((uint16_t*)job.out)[at] = job.out_dt == DT_F16 ? f32_to_f16(x) : f32_to_bf16(x);
            }
        }
    }
}

// the splits' sums in split order, 4 elements a thread (a job's count is a multiple of 8)
__global__ __launch_bounds__(256) void tokens_join_kernel(TokenLaunch p) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= p.total) return;
    f32x4 v = *(const f32x4*)(p.partial + i);
    for (int s = 1; s < p.splits; ++s) v += *(const f32x4*)(p.partial + s * p.total + i);
    int k = p.jobs - 1;
    while (k > 0 && i < p.at[k]) --k;
    const TokenJob job = p.job[k];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t at = i - p.at[k] + e;
        const float x = v[e] * job.post;
        if (job.out_dt == DT_F32) ((float*)job.out)[at] = x;
        else ((uint16_t*)job.out)[at] = job.out_dt == DT_F16 ? f32_to_f16(x) : f32_to_bf16(x);
    }
}

static int64_t token_tiles(int64_t C) { return (C + TK_C - 1) / TK_C; }

// About four workgroups a CU (two at a time), at least 8 steps each, at most 8 splits
int tokens_splits(int64_t M, int64_t tiles) {
    const int64_t steps = (M + TK_T - 1) / TK_T;
    if (tiles <= 0) return 1;
    int64_t s = (4 * device_rates().cus + tiles - 1) / tiles;
    if (s > steps / 8) s = steps / 8;
    if (s > 8) s = 8;
    return s > 1 ? (int)s : 1;
}

size_t tokens_partial(int64_t M, int64_t K, int64_t N, int64_t r, bool dd, bool du) {
    const int64_t tiles = (dd ? 2 * token_tiles(K) : 0) + (du ? 2 * token_tiles(N) : 0);
    const int s = tokens_splits(M, tiles);
    return s > 1 ? (size_t)s * (size_t)((dd ? 2 * K : 0) + (du ? 2 * N : 0)) * (size_t)r * 4 : 0;
}

template <class CT>
static hipError_t run_tokens(const TokenLaunch& p, int64_t r, hipStream_t s) {
    const dim3 g((unsigned)p.end[p.jobs - 1], (unsigned)p.splits);
    if (r <= 64) hipLaunchKernelGGL((tokens_kernel<CT, 64>), g, dim3(256), 0, s, p);
    else if (r <= 128) hipLaunchKernelGGL((tokens_kernel<CT, 128>), g, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((tokens_kernel<CT, 256>), g, dim3(256), 0, s, p);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.splits > 1) {
        hipLaunchKernelGGL(tokens_join_kernel, dim3((unsigned)((p.total / 4 + 255) / 256)), dim3(256), 0, s, p);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_tokens(int c_dt, const TokenJob* jobs, int n, int64_t M, float* partial, hipStream_t s) {
    TokenLaunch p{};
    if (n < 1 || n > 4) return hipErrorInvalidValue;
    int64_t tiles = 0;
    for (int i = 0; i < n; ++i) {
        const TokenJob& j = jobs[i];
        if (j.C % 8 != 0 || j.r < 1 || j.r > 256 || j.r != jobs[0].r || j.ldr % 8 != 0 ||
            M * j.C * 2 >= ((int64_t)1 << 30) || M * j.ldr * 2 > ((int64_t)1 << 30))   // (the longest batch: h's rows at 1 GiB)
            return hipErrorInvalidValue;
        p.job[i] = j;
        p.at[i] = p.total;
        p.total += j.C * j.r;
        tiles += token_tiles(j.C);
        p.end[i] = (int)tiles;
    }
    if (tiles == 0) return hipSuccess;
    p.M = M;
    p.jobs = n;
    p.splits = tokens_splits(M, tiles);
    p.partial = partial;
    if (p.splits > 1 && partial == nullptr) return hipErrorInvalidValue;
    return c_dt == DT_F16 ? run_tokens<CF16>(p, jobs[0].r, s) : run_tokens<CBF16>(p, jobs[0].r, s);
}

}  // namespace lyc
