// mx_rows.cu -- row operators that end in microscaled codes:
//
//  * rmsnorm_kernel: the residual's addition, the root-mean-square norm and
//    its output, once in the input's type and once as e4m3 codes with a scale
//    per 32 columns:
//      s = round(h + delta)          (h, when there is no delta)
//      n_i = s_i * (mean_j s_j^2 + eps)^(-1/2) * w_i
//      y = round(n), (q, scale) = MX(n)
//  * quantize_kernel: (q, scale) = MX(x), and optionally the values that the
//    codes stand for, in x's type.
//
// Both read every input once and write every output once, and are bound by
// that: the norm of 16384 x 4096 bf16 rows with an fp32 delta and every output
// takes 110 us (6.7 TB/s; 113 us in long runs), the quantisation of 114688 x
// 4096 bf16 values to e2m1 with their values written back 314 us (6.8 TB/s;
// 350 us in long runs, at a clock that the power cap lowers), 4097 x 4096 to
// e4m3 10 us (in L2), one row of 4096 2.4 us, the latency of a launch and of
// two rounds through memory.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"

namespace moe {

namespace {

struct NormParams {
    int d, nvec, pitch;
    const uint8_t *h, *delta, *w;
    long long h_stride, delta_stride;  // bytes
    float eps;
    uint8_t *h_out, *y, *q, *scales;   // any may be null (q and scales together)
    long long q_stride, s_stride;      // bytes
};

constexpr int kDeltaNone = 0, kDeltaSame = 1, kDeltaFp32 = 2;

// The scale byte of the block that lanes 4i..4i+3 hold eight values each of.
template <int FMT>
__device__ __forceinline__ uint32_t block_code(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return mx_scale_code<FMT>(m);
}

// One CTA per row, V vectors of eight values per thread, held in registers
// between the sum and the outputs, so a row is read once.  Long runs are held
// by the power cap, and two vectors a thread do the same loads with less
// (16384 x 4096: one vector 123 us, two 113, four 115).  The squares are summed in fp64: the conversions hide behind the
// loads, and the statistic is right for every input, also one whose squares
// leave fp32's range.
template <int TYPE, int DELTA, int V>
__global__ void rmsnorm_kernel(const NormParams p)
{
    __shared__ double part[32];
    ptx::grid_dep_launch();
    const int tid = threadIdx.x;
    const size_t row = blockIdx.x;
    constexpr int kBytes = 8 * type_size<TYPE>();
    constexpr int DT = DELTA == kDeltaFp32 ? kTypeFp32 : TYPE;
    Vec8<TYPE> hv[V];
    Vec8<DT> dv[V];
    ptx::grid_dep_wait();
    const uint8_t *hr = p.h + row * p.h_stride;
    const uint8_t *dr = DELTA == kDeltaNone ? nullptr : p.delta + row * p.delta_stride;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int i = tid + u * blockDim.x;
        if (i < p.nvec) {
            hv[u] = load8<TYPE>(hr + static_cast<size_t>(i) * kBytes);
            if constexpr (DELTA != kDeltaNone)
                dv[u] = load8<DT>(dr + static_cast<size_t>(i) * 8 * type_size<DT>());
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int i = tid + u * blockDim.x;
        if (i < p.nvec) {
            float v[8];
            unpack8<TYPE>(hv[u], v);
            if constexpr (DELTA != kDeltaNone) {
                float a[8];
                unpack8<DT>(dv[u], a);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += a[j];
                // the norm is of the stream as it is stored
                hv[u] = pack8<TYPE>(v);
                unpack8<TYPE>(hv[u], v);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double x = v[j];
                sum = fma(x, x, sum);
            }
            if (p.h_out)
                store8<TYPE>(p.h_out + (row * p.nvec + i) * kBytes, hv[u]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((tid & 31) == 0) part[tid >> 5] = sum;
    __syncthreads();
    const int warps = blockDim.x >> 5;
    sum = (tid & 31) < warps ? part[tid & 31] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = static_cast<float>(1.0 / sqrt(sum / p.d + static_cast<double>(p.eps)));
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int i = tid + u * blockDim.x;
        const bool has = i < p.nvec;
        float v[8];
        if (has) {
            float w[8];
            unpack8<TYPE>(hv[u], v);
            unpack8<TYPE>(load8<TYPE>(p.w + static_cast<size_t>(i) * kBytes), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = v[j] * r * w[j];
            if (p.y) store8<TYPE>(p.y + (row * p.nvec + i) * kBytes, pack8<TYPE>(v));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
        if (p.q) {
            const uint32_t c = block_code<kMxE4M3>(v);
            if (has) {
                *reinterpret_cast<uint2 *>(p.q + row * p.q_stride + static_cast<size_t>(i) * 8) =
                    mx_codes8<kMxE4M3>(v, c);
                if ((i & 3) == 0) p.scales[row * p.s_stride + (i >> 2)] = static_cast<uint8_t>(c);
            }
        }
    }
    if (p.q && tid < p.pitch - (p.nvec >> 2))
        p.scales[row * p.s_stride + (p.nvec >> 2) + tid] = 0;
}

struct QuantParams {
    uint32_t total, nvec;  // vectors of eight in all, and per row
    uint32_t step_row, step_col;  // kQuantThreads vectors on, in rows and columns
    int pitch;
    const uint8_t *x;
    long long x_stride;    // bytes
    uint8_t *q, *scales, *hat;
};

constexpr int kQuantThreads = 256;
constexpr int kQuantVec = 4;  // vectors per thread, loads in flight together

template <int TYPE, int FMT, bool HAT>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantParams p)
{
    ptx::grid_dep_launch();
    constexpr int kBytes = 8 * type_size<TYPE>();
    constexpr int kCode = FMT == kMxE4M3 ? 8 : 4;
    const uint32_t base = blockIdx.x * (kQuantThreads * kQuantVec) + threadIdx.x;
    Vec8<TYPE> xv[kQuantVec];
    // One division a thread: 351 us instead of 357 for 114688 x 4096 in long
    // runs, which the power cap holds.
    uint32_t row[kQuantVec], col[kQuantVec];
    row[0] = base / p.nvec;
    col[0] = base - row[0] * p.nvec;
#pragma unroll
    for (int u = 1; u < kQuantVec; ++u) {
        row[u] = row[u - 1] + p.step_row;
        col[u] = col[u - 1] + p.step_col;
        if (col[u] >= p.nvec) {
            col[u] -= p.nvec;
            ++row[u];
        }
    }
    ptx::grid_dep_wait();
#pragma unroll
    for (int u = 0; u < kQuantVec; ++u) {
        const uint32_t i = base + u * kQuantThreads;
        if (i < p.total)
            xv[u] = load8<TYPE>(p.x + row[u] * p.x_stride + static_cast<size_t>(col[u]) * kBytes);
    }
#pragma unroll
    for (int u = 0; u < kQuantVec; ++u) {
        const uint32_t i = base + u * kQuantThreads;
        const bool has = i < p.total;  // the same for the four lanes of a block
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (has) unpack8<TYPE>(xv[u], v);
        const uint32_t c = block_code<FMT>(v);
        if (!has) continue;
        const uint2 q = mx_codes8<FMT>(v, c);
        if constexpr (FMT == kMxE4M3) *reinterpret_cast<uint2 *>(p.q + static_cast<size_t>(i) * kCode) = q;
        else *reinterpret_cast<uint32_t *>(p.q + static_cast<size_t>(i) * kCode) = q.x;
        if ((col[u] & 3) == 0) {
            uint8_t *s = p.scales + static_cast<size_t>(row[u]) * p.pitch;
            s[col[u] >> 2] = static_cast<uint8_t>(c);
            if (col[u] == p.nvec - 4)
                for (int b = static_cast<int>(p.nvec >> 2); b < p.pitch; ++b) s[b] = 0;
        }
        if constexpr (HAT) {
            mx_values8<FMT>(q, c, v);
            store8<TYPE>(p.hat + static_cast<size_t>(i) * kBytes, pack8<TYPE>(v));
        }
    }
}

template <int TYPE, int DELTA>
cudaError_t norm_v(const NormParams &p, int T, cudaStream_t s, bool pdl)
{
    const int v = p.nvec <= 256 ? 1 : p.nvec <= 1024 ? 2 : 4;
    const int thr = ((p.nvec + v - 1) / v + 31) / 32 * 32;
    auto *k = v == 1 ? rmsnorm_kernel<TYPE, DELTA, 1>
              : v == 2 ? rmsnorm_kernel<TYPE, DELTA, 2> : rmsnorm_kernel<TYPE, DELTA, 4>;
    return launch_pdl(k, dim3(T), dim3(thr), 0, s, pdl, p);
}

template <int TYPE>
cudaError_t norm_t(const NormParams &p, int T, int delta, cudaStream_t s, bool pdl)
{
    if (delta == kDeltaNone) return norm_v<TYPE, kDeltaNone>(p, T, s, pdl);
    if (delta == kDeltaSame) return norm_v<TYPE, kDeltaSame>(p, T, s, pdl);
    if constexpr (TYPE == kTypeFp32) return cudaErrorInvalidValue;
    else return norm_v<TYPE, kDeltaFp32>(p, T, s, pdl);
}

template <int TYPE>
cudaError_t quant_t(const QuantParams &p, int fmt, cudaStream_t s, bool pdl)
{
    auto *k = fmt == kMxE4M3
                  ? (p.hat ? quantize_kernel<TYPE, kMxE4M3, true> : quantize_kernel<TYPE, kMxE4M3, false>)
                  : (p.hat ? quantize_kernel<TYPE, kMxE2M1, true> : quantize_kernel<TYPE, kMxE2M1, false>);
    const uint32_t per = kQuantThreads * kQuantVec;
    return launch_pdl(k, dim3((p.total + per - 1) / per), dim3(kQuantThreads), 0, s, pdl, p);
}

int size_of(int type) { return type == kTypeFp32 ? 4 : 2; }

}  // namespace

cudaError_t launch_rmsnorm(const NormLaunch &a, cudaStream_t s)
{
    NormParams p{};
    p.d = a.d;
    p.nvec = a.d / 8;
    p.pitch = mx_scale_pitch(a.d);
    p.h = static_cast<const uint8_t *>(a.h);
    p.delta = static_cast<const uint8_t *>(a.delta);
    p.w = static_cast<const uint8_t *>(a.w);
    p.h_stride = a.h_stride * size_of(a.type);
    p.delta_stride = a.delta_stride * size_of(a.delta_type);
    p.eps = a.eps;
    p.h_out = static_cast<uint8_t *>(a.h_out);
    p.y = static_cast<uint8_t *>(a.y);
    p.q = a.q;
    p.scales = a.scales;
    p.q_stride = a.q_stride;
    p.s_stride = a.s_stride;
    const int delta = a.delta == nullptr ? kDeltaNone : a.delta_type == a.type ? kDeltaSame : kDeltaFp32;
    if (a.type == kTypeBf16) return norm_t<kTypeBf16>(p, a.T, delta, s, a.pdl);
    if (a.type == kTypeFp16) return norm_t<kTypeFp16>(p, a.T, delta, s, a.pdl);
    return norm_t<kTypeFp32>(p, a.T, delta, s, a.pdl);
}

cudaError_t launch_mx_quantize(const MxQuantLaunch &a, cudaStream_t s)
{
    QuantParams p{};
    p.nvec = static_cast<uint32_t>(a.cols / 8);
    p.total = static_cast<uint32_t>(a.rows) * p.nvec;
    p.step_row = kQuantThreads / p.nvec;
    p.step_col = kQuantThreads % p.nvec;
    p.pitch = mx_scale_pitch(a.cols);
    p.x = static_cast<const uint8_t *>(a.x);
    p.x_stride = a.x_stride * size_of(a.type);
    p.q = a.q;
    p.scales = a.scales;
    p.hat = static_cast<uint8_t *>(a.hat);
    if (a.type == kTypeBf16) return quant_t<kTypeBf16>(p, a.fmt, s, a.pdl);
    if (a.type == kTypeFp16) return quant_t<kTypeFp16>(p, a.fmt, s, a.pdl);
    return quant_t<kTypeFp32>(p, a.fmt, s, a.pdl);
}

}  // namespace moe
