// gate.cuh -- the experts' gate: silu(g) * b (act 0) or sigmoid(g) * b (act 1),
// sigmoid(g) = 1 / (1 + exp(-g)).
//
// gate_mul() is one division, g * b / (1 + exp(-g)), which holds while g * b
// and exp(-g) stay below 2^126; beyond, it gives NaN (g = -1e20, b = 1e20: the
// gate is 0), infinity (g = -50, b = 1e38) or 0 (g = -88).  `most` keeps the
// largest of both over a thread's calls, for one test behind them: the values
// of a chunk that reached kGateRange are computed again with gate_redo(), one
// at a time, and the chunks that did not pay one vote.  (A branch at every
// value instead: 4096 tokens of d = 512, d_ff = 1024 82 us, this way 80 us.
// gate_redo()'s second form for every value: 8192 microscaled rows of 4096 ->
// 2 x 14336 773 us, this way 747 us.)
//
// Exponential and division are CUDA's fast ones, which are off by a few 2^-23
// (the exponential by |g| 2^-24 more).  7.4e7 e4m3 values of 4096 -> 2 x 4096, of
// which those count that are not the ones of 64 bits: 87 on e4m3 rows and 52 on
// e2m1 rows; with rounded functions on the same sums 80 and 57, and the gated
// prefill product 12 % slower.
#pragma once

namespace moe {

constexpr float kGateRange = 0x1p126f;

__device__ __forceinline__ float gate_mul(float g, float b, int act, float &most)
{
    const float num = act ? b : g * b;
    const float den = 1.0f + __expf(-g);
    most = fmaxf(most, fmaxf(fabsf(num), den));
    return __fdividef(num, den);
}

// gate_mul()'s value where it holds, bit for bit.  Elsewhere, with
// h = exp(-|g| / 2),
//   act(g) * b = (g / (1 + h^2)) * b            g >= 0
//              = (h * g / (1 + h^2)) * (h * b)  g < 0
// no step of which leaves fp32's range unless the result does.
__device__ __forceinline__ float gate_redo(float g, float b, int act)
{
    float most = 0.0f;
    const float v = gate_mul(g, b, act, most);
    if (most < kGateRange) return v;
    const float h = __expf(-0.5f * fabsf(g));
    const float a = g < 0.0f ? h : 1.0f;
    return __fdividef(act ? a : a * g, 1.0f + h * h) * (a * b);
}

}  // namespace moe
