// Backward pass of the RMS norm with a residual stream, for gfx950.
//
// The forward pass (rmsnorm_quant_kernel) normalizes rows h, y = h r w with r = 1 / sqrt(mean(h^2) + eps), and hands h on
// as the residual stream.  With dy the gradient of y (from DGrad) and dres that of h by way of the stream, and the
// roundings of y and of its codes taken as the identity:
//   g = dy w,   dx = r (g - h r^2 mean(g h)) + dres,   dw = sum over the rows of dy h r.
// Gradients between operators stay bf16 (Jet-RL explainers, "Schema de Quantification"); the row sums, the column sums
// and dw are fp32 or wider.
#include "jetfp8_common.h"
#include "jetfp8_launch.h"

namespace jetfp8 {

namespace {

struct NormBackArgs {
    const uint16_t *dy, *h, *w;
    const float* rstd;
    const uint16_t* dres;      // may be null
    uint16_t* dx;
    float* part;               // column sums of each thread block, [blocks][C]; null: dw is not wanted
    int64_t rows, cols;
};

// A team of WPR waves takes a row, TEAMS of them in a thread block take rows in turn.  A wave's k-th chunk covers 512
// columns, lane l columns 8 l .. + 7 of it, as in the forward kernel; what a lane holds of dy, h and dres is loaded once,
// the row's sum meets in LDS (two buffers, so one barrier a row), and each lane keeps the column sums of its columns in
// registers over all rows of its thread block.  h enters as h r alone, whose size is that of 1: g h overflows fp32 and r^2
// underflows for rows that bf16 and the forward pass still hold.
template <int HCH, int WPR, int TEAMS>
__global__ __launch_bounds__(WPR * TEAMS * 64) void rmsnorm_backward_kernel(NormBackArgs a) {
    __shared__ float sums[2][TEAMS][WPR];
    __shared__ float cols[TEAMS > 1 ? WPR * HCH * 512 : 1];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int team = wave / WPR, part = wave % WPR;
    const float inv_cols = 1.0f / (float)a.cols;
    int64_t col[HCH];
    bool ok[HCH];
    uint4 w[HCH];
    float dw[HCH][8];
#pragma unroll
    for (int k = 0; k < HCH; ++k) {
        col[k] = (int64_t)(part * HCH + k) * 512 + lane * 8;
        ok[k] = col[k] < a.cols;
        w[k] = make_uint4(0, 0, 0, 0);
        if (ok[k]) w[k] = ld16(a.w + col[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
    }
    // every team of a thread block makes the same number of turns (the barrier); one without a row computes zeros
    int buf = 0;
    for (int64_t first = (int64_t)blockIdx.x * TEAMS; first < a.rows; first += (int64_t)gridDim.x * TEAMS, buf ^= 1) {
        const int64_t row = first + team;
        const bool live = row < a.rows;
        uint4 dy[HCH], h[HCH], dr[HCH];
#pragma unroll
        for (int k = 0; k < HCH; ++k) {
            dy[k] = h[k] = dr[k] = make_uint4(0, 0, 0, 0);
            if (live && ok[k]) {
                const int64_t at = row * a.cols + col[k];
                dy[k] = ld16(a.dy + at);
                h[k] = ld16(a.h + at);
                if (a.dres) dr[k] = ld16(a.dres + at);
            }
        }
        const float r = live ? a.rstd[row] : 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < HCH; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum = fmaf(elem_of(dy[k], i) * elem_of(w[k], i), elem_of(h[k], i) * r, sum);
        sum = wave_sum(sum);
        if (WPR > 1) {
            if (lane == 0) sums[buf][team][part] = sum;
            __syncthreads();
            sum = sums[buf][team][0];
#pragma unroll
            for (int p = 1; p < WPR; ++p) sum += sums[buf][team][p];
        }
        const float mean = sum * inv_cols;
#pragma unroll
        for (int k = 0; k < HCH; ++k) {
            float out[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = elem_of(dy[k], i), n = elem_of(h[k], i) * r;
                out[i] = fmaf(r, fmaf(-n, mean, y * elem_of(w[k], i)), elem_of(dr[k], i));
                dw[k][i] = fmaf(y, n, dw[k][i]);
            }
            if (live && ok[k]) *reinterpret_cast<uint4*>(a.dx + row * a.cols + col[k]) = bf16x8_rne(out);
        }
    }
    if (!a.part) return;
    // the teams' column sums, added in team order
#pragma unroll
    for (int t = 1; t < TEAMS; ++t) {
        __syncthreads();
        if (team == t) {
#pragma unroll
            for (int k = 0; k < HCH; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) cols[((part * HCH + k) * 8 + i) * 64 + lane] = dw[k][i];
        }
        __syncthreads();
        if (team == 0) {
#pragma unroll
            for (int k = 0; k < HCH; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[k][i] += cols[((part * HCH + k) * 8 + i) * 64 + lane];
        }
    }
    if (team) return;
#pragma unroll
    for (int k = 0; k < HCH; ++k)
        if (ok[k]) {
            float* to = a.part + (int64_t)blockIdx.x * a.cols + col[k];
            *reinterpret_cast<float4*>(to) = make_float4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
            *reinterpret_cast<float4*>(to + 4) = make_float4(dw[k][4], dw[k][5], dw[k][6], dw[k][7]);
        }
}

// dw from the thread blocks' column sums, added in fp64 in a fixed order: 64 columns to a thread block, each of its 64
// groups of 16 lanes takes every 64th part (512 parts of 4096 columns with 16 groups: 10 us).
constexpr int kWeightGroups = 64;
__global__ __launch_bounds__(kWeightGroups * 16) void norm_weight_kernel(const float* __restrict__ part, int parts,
                                                                         int64_t cols, float* __restrict__ dw) {
    __shared__ double all[kWeightGroups][64];
    const int lane = threadIdx.x % 16, group = threadIdx.x / 16;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane * 4;
    double s[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (int p = group; p < parts; p += kWeightGroups) {
        const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)p * cols + col);
        s[0] += v.x;
        s[1] += v.y;
        s[2] += v.z;
        s[3] += v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) all[group][lane * 4 + i] = s[i];
    __syncthreads();
    // 16 partial sums of each column, then those
    const int column = threadIdx.x % 64, part16 = threadIdx.x / 64;
    double t = 0;
#pragma unroll
    for (int g = 0; g < kWeightGroups / 16; ++g) t += all[part16 * (kWeightGroups / 16) + g][column];
    __syncthreads();
    all[part16][column] = t;
    __syncthreads();
    if (threadIdx.x < 64) {
        t = 0;
#pragma unroll
        for (int g = 0; g < 16; ++g) t += all[g][column];
        dw[(int64_t)blockIdx.x * 64 + column] = (float)t;
    }
}

constexpr int64_t kNormBackBlocks = 512;

template <int HCH, int WPR, int TEAMS>
hipError_t launch(const NormBackArgs& a, int64_t blocks, hipStream_t st) {
    rmsnorm_backward_kernel<HCH, WPR, TEAMS><<<(unsigned)blocks, WPR * TEAMS * 64, 0, st>>>(a);
    return hipGetLastError();
}

int64_t back_blocks(int64_t R) {
    const int64_t n = (R + 1) / 2;
    return n < kNormBackBlocks ? n : kNormBackBlocks;
}

}  // namespace

int64_t rmsnorm_backward_workspace(int64_t R, int64_t C) { return back_blocks(R) * C * (int64_t)sizeof(float); }

hipError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* w, const float* rstd,
                                   const uint16_t* dres, int64_t R, int64_t C, uint16_t* dx, float* dw, float* workspace,
                                   hipStream_t st) {
    const NormBackArgs a{dy, h, w, rstd, dres, dx, dw ? workspace : nullptr, R, C};
    const int64_t blocks = back_blocks(R);
    const int nch = (int)((C + 511) / 512);
    hipError_t e;
    if (nch <= 1) e = launch<1, 1, 2>(a, blocks, st);
    else if (nch <= 2) e = launch<2, 1, 2>(a, blocks, st);
    else if (nch <= 4) e = launch<2, 2, 2>(a, blocks, st);
    else if (nch <= 6) e = launch<2, 3, 2>(a, blocks, st);
    else if (nch <= 8) e = launch<2, 4, 2>(a, blocks, st);
    else if (nch <= 10) e = launch<2, 5, 2>(a, blocks, st);
    else if (nch <= 12) e = launch<3, 4, 2>(a, blocks, st);
    else e = launch<4, 4, 2>(a, blocks, st);
    if (e != hipSuccess || !dw) return e;
    norm_weight_kernel<<<(unsigned)(C / 64), kWeightGroups * 16, 0, st>>>(workspace, (int)blocks, C, dw);
    return hipGetLastError();
}

}  // namespace jetfp8
