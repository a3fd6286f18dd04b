// mx_gemm.cu -- products of microscaled rows with 4-bit expert weights:
//   y[r, n] = sum_k W_e[n, k] x[r, k]                   (moe_mx_product)
//   h[r, f] = act(W1_e x[r])[f] * (W3_e x[r])[f]        (moe_mx_gated)
// for every row r of expert e's segment, x in e4m3 or e2m1, W in e2m1, one
// power-of-two scale per 32 values of K on both sides, sums in fp32.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"

namespace moe {

namespace {

struct GemmParams {
    int S, K, E, N, act, y_type;
    const uint8_t *x, *xs, *W1, *s1, *W3, *s3;
    long long x_stride, xs_stride;
    const int32_t *offsets;
    void *y;
    uint8_t *q, *qs;
    uint32_t *err;
};

constexpr int kTile = 64;

template <int FMT>
__device__ void load_tile(float (*dst)[33], const uint8_t *q, long long qst, const uint8_t *s,
                          long long sst, int r0, int rows, int k0)
{
    // 64 rows x 32 values: thread t reads eight values of row t / 4.
    const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r0 + r < rows) {
        const uint8_t *p = q + (r0 + r) * qst;
        uint2 w;
        if constexpr (FMT == kMxE4M3) w = *reinterpret_cast<const uint2 *>(p + k0 + c);
        else w = make_uint2(*reinterpret_cast<const uint32_t *>(p + (k0 + c) / 2), 0u);
        mx_values8<FMT>(w, s[(r0 + r) * sst + k0 / 32], v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[r][c + i] = v[i];
}

template <int FMT, bool GATED>
__global__ void __launch_bounds__(256) mx_gemm_kernel(const GemmParams p)
{
    __shared__ float sx[kTile][33], sw[kTile][33], sv[GATED ? kTile : 1][33];
    __shared__ float sh[GATED ? kTile : 1][kTile + 1];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int tid = threadIdx.x;
    bool bad = false;
    for (int e = tid; e < p.E; e += 256)
        if (p.offsets) {
            const int a = p.offsets[e], b = p.offsets[e + 1];
            bad |= a < 0 || b < a || b > p.S;
        }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(p.err, kErrOffsets);
        return;
    }
    const int e = blockIdx.y, n0 = blockIdx.x * kTile;
    const int first = p.offsets ? p.offsets[e] : 0, last = p.offsets ? p.offsets[e + 1] : p.S;
    const size_t wrow = static_cast<size_t>(e) * p.N;
    const int wp = p.K / 2, sp = mx_scale_pitch(p.K);
    const uint8_t *W1 = p.W1 + wrow * wp, *s1 = p.s1 + wrow * sp;
    const uint8_t *W3 = GATED ? p.W3 + wrow * wp : nullptr, *s3 = GATED ? p.s3 + wrow * sp : nullptr;
    const int tr = tid >> 4, tc = tid & 15;
    for (int r0 = first; r0 < last; r0 += kTile) {
        float a[4][4] = {}, b[4][4] = {};
        for (int k0 = 0; k0 < p.K; k0 += 32) {
            load_tile<FMT>(sx, p.x, p.x_stride, p.xs, p.xs_stride, r0, last, k0);
            load_tile<kMxE2M1>(sw, W1, wp, s1, sp, n0, p.N, k0);
            if constexpr (GATED) load_tile<kMxE2M1>(sv, W3, wp, s3, sp, n0, p.N, k0);
            __syncthreads();
            for (int k = 0; k < 32; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) {
                        a[i][j] = fmaf(sx[tr + 16 * i][k], sw[tc + 16 * j][k], a[i][j]);
                        if constexpr (GATED) b[i][j] = fmaf(sx[tr + 16 * i][k], sv[tc + 16 * j][k], b[i][j]);
                    }
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int r = r0 + tr + 16 * i, n = n0 + tc + 16 * j;
                float v = a[i][j];
                if constexpr (GATED) {
                    const float g = v;
                    v = (p.act ? 1.0f : g) * b[i][j] / (1.0f + expf(-g));
                    sh[tr + 16 * i][tc + 16 * j] = v;
                }
                if (p.y && r < last && n < p.N) {
                    const size_t at = static_cast<size_t>(r) * p.N + n;
                    if (p.y_type == kTypeBf16) static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v);
                    else static_cast<float *>(p.y)[at] = v;
                }
            }
        if constexpr (GATED) {
            __syncthreads();
            const int r = r0 + (tid >> 2), c = (tid & 3) * 16;
            if (p.q) {
                // two threads a block of 32 columns, sixteen values each
                uint32_t m = 0;
                for (int i = 0; i < 16; ++i) m = max(m, abs_bits(sh[tid >> 2][c + i]));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                const uint32_t code = mx_scale_code<kMxE4M3>(m);
                if (r < last && n0 + c < p.N) {
                    for (int o = 0; o < 16; o += 8) {
                        float v[8];
                        for (int i = 0; i < 8; ++i) v[i] = sh[tid >> 2][c + o + i];
                        *reinterpret_cast<uint2 *>(p.q + static_cast<size_t>(r) * p.N + n0 + c + o) =
                            mx_codes8<kMxE4M3>(v, code);
                    }
                    uint8_t *s = p.qs + static_cast<size_t>(r) * mx_scale_pitch(p.N);
                    if ((tid & 1) == 0) s[(n0 + c) / 32] = static_cast<uint8_t>(code);
                    if (n0 + c + 16 == p.N)
                        for (int b = p.N / 32; b < mx_scale_pitch(p.N); ++b) s[b] = 0;
                }
            }
            __syncthreads();
        }
    }
}

}  // namespace

size_t mx_gemm_zero_bytes(int, int, int) { return 0; }
size_t mx_gemm_scratch_bytes(int, int, int) { return 0; }

cudaError_t launch_mx_gemm(const MxGemmLaunch &a, cudaStream_t s)
{
    GemmParams p{};
    p.S = a.S;
    p.K = a.K;
    p.E = a.E;
    p.N = a.N;
    p.act = a.act;
    p.y_type = a.y_type;
    p.x = a.x;
    p.xs = a.xs;
    p.x_stride = a.x_stride;
    p.xs_stride = a.xs_stride;
    p.W1 = a.W1;
    p.s1 = a.s1;
    p.W3 = a.W3;
    p.s3 = a.s3;
    p.offsets = a.offsets;
    p.y = a.y;
    p.q = a.q;
    p.qs = a.qs;
    p.err = a.err;
    auto *k = a.fmt == kMxE4M3 ? (a.W3 ? mx_gemm_kernel<kMxE4M3, true> : mx_gemm_kernel<kMxE4M3, false>)
                               : (a.W3 ? mx_gemm_kernel<kMxE2M1, true> : mx_gemm_kernel<kMxE2M1, false>);
    return launch_pdl(k, dim3((a.N + kTile - 1) / kTile, a.E), dim3(256), 0, s, a.pdl, p);
}

}  // namespace moe
