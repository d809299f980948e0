// epilogue.cuh -- what follows a W4A16 product before its single rounding to
// binary16: bias, activation, gate, residual.
//
//   t[m, n] = sum_k X'[m, k] w[k, n] + bias[n]               (float)
//   a[m, n] = act(t[m, n])                                    or, gated,
//   a[m, j] = act(t[m, 2j]) * t[m, 2j + 1]                    (N / 2 columns)
//   Y       = binary16_RNE(a + residual)
//
// The matmul kernels are instantiated twice, with and without it: the plain
// instantiations hold none of this code.  The accumulators are read where the
// plain kernel rounds them, so the bias, the activation and the residual cost
// their own bytes (2 N + 2 M N) and no further pass over Y.
#pragma once

#include <type_traits>

#include "awq_common.cuh"

namespace awq {

struct Epilogue {
    const __half *bias;      // [N] or NULL
    const __half *residual;  // [M, columns of Y] or NULL; may be Y itself
    int act;                 // awq_act_t
    int gated;               // columns 2j are the gate of columns 2j + 1
};

// Activation in float.  The exponentials use the fast forms (a few units of
// 2^-22 relative), far below the binary16 rounding that follows.
__device__ __forceinline__ float epi_sigmoid_times(float t, float u)  // t * sigmoid(u)
{
    return __fdividef(t, 1.0f + __expf(-u));
}

template <int ACT>
__device__ __forceinline__ float epi_act_of(float t)
{
    if constexpr (ACT == AWQ_ACT_RELU) return t < 0.0f ? 0.0f : t;  // NaN stays NaN
    if constexpr (ACT == AWQ_ACT_SILU) return epi_sigmoid_times(t, t);
    if constexpr (ACT == AWQ_ACT_GELU) return 0.5f * t * erfcf(-0.70710678f * t);
    // 0.5 t (1 + tanh(u)) = t sigmoid(2u), u = sqrt(2/pi) (t + 0.044715 t^3)
    if constexpr (ACT == AWQ_ACT_GELU_TANH) return epi_sigmoid_times(t, 1.59576912f * (t + 0.044715f * t * t * t));
    return t;
}

// f(integral_constant<int, act>): the choice is made once per call, not per
// value.  (Inside unrolled loops it multiplied the code by the five activations:
// the prompt kernels then ran out of the instruction cache, and a bias alone
// took 2048 x 4096 x 28672 from 424 to 526 us, a gate to 691.)
template <class F>
__device__ __forceinline__ void epi_with_act(int act, F &&f)
{
    switch (act) {
    case AWQ_ACT_RELU: f(std::integral_constant<int, AWQ_ACT_RELU>{}); break;
    case AWQ_ACT_SILU: f(std::integral_constant<int, AWQ_ACT_SILU>{}); break;
    case AWQ_ACT_GELU: f(std::integral_constant<int, AWQ_ACT_GELU>{}); break;
    case AWQ_ACT_GELU_TANH: f(std::integral_constant<int, AWQ_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, AWQ_ACT_NONE>{}); break;
    }
}

__device__ __forceinline__ float epi_act(float t, int act)
{
    epi_with_act(act, [&](auto a) { t = epi_act_of<decltype(a)::value>(t); });
    return t;
}

__device__ __forceinline__ float epi_bias(const Epilogue &e, int n)
{
    return e.bias ? __half2float(e.bias[n]) : 0.0f;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    return __half_as_ushort(__float2half_rn(lo)) | (static_cast<uint32_t>(__half_as_ushort(__float2half_rn(hi))) << 16);
}

__device__ __forceinline__ float half_lo(uint32_t w) { return __half2float(__ushort_as_half(static_cast<uint16_t>(w))); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16))); }

// What columns n .. n + 7 of token `tok` (N columns before the gate) need
// besides their sums; zeros where the call has none.
struct Epi8 {
    uint4 bias, residual;  // gated: four residuals, in x and y
};

__device__ __forceinline__ Epi8 epi_load8(const Epilogue &e, int tok, int n, int N)
{
    Epi8 x{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (e.bias) x.bias = *reinterpret_cast<const uint4 *>(e.bias + n);
    if (e.residual && e.gated) {
        const uint2 r = *reinterpret_cast<const uint2 *>(e.residual + static_cast<size_t>(tok) * (N / 2) + n / 2);
        x.residual.x = r.x;
        x.residual.y = r.y;
    } else if (e.residual) {
        x.residual = *reinterpret_cast<const uint4 *>(e.residual + static_cast<size_t>(tok) * N + n);
    }
    return x;
}

// Finishes and writes those eight columns, 16 bytes, or 8 bytes when gated.
__device__ __forceinline__ void epi_store8(const Epilogue &e, const Epi8 &x, float (&v)[8], __half *Y, int tok, int n,
                                           int N)
{
    if (e.bias) {
        const uint32_t w[4] = {x.bias.x, x.bias.y, x.bias.z, x.bias.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] += half_lo(w[i]);
            v[2 * i + 1] += half_hi(w[i]);
        }
    }
    if (e.gated) {
        epi_with_act(e.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = epi_act_of<decltype(a)::value>(v[2 * i]) * v[2 * i + 1];
        });
        const size_t at = static_cast<size_t>(tok) * (N / 2) + n / 2;
        if (e.residual) {
            const uint4 r = x.residual;
            v[0] += half_lo(r.x); v[1] += half_hi(r.x); v[2] += half_lo(r.y); v[3] += half_hi(r.y);
        }
        *reinterpret_cast<uint2 *>(Y + at) = make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
        return;
    }
    epi_with_act(e.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = epi_act_of<decltype(a)::value>(v[i]);
    });
    const size_t at = static_cast<size_t>(tok) * N + n;
    if (e.residual) {
        const uint32_t w[4] = {x.residual.x, x.residual.y, x.residual.z, x.residual.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] += half_lo(w[i]);
            v[2 * i + 1] += half_hi(w[i]);
        }
    }
    *reinterpret_cast<uint4 *>(Y + at) = make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]),
                                                    pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
}

__device__ __forceinline__ void epi_store8(const Epilogue &e, float (&v)[8], __half *Y, int tok, int n, int N)
{
    epi_store8(e, epi_load8(e, tok, n, N), v, Y, tok, n, N);
}

// The residual of token `tok`, columns n0 .. n0 + 127 before the gate, on its way
// into L2 while the products run: the epilogue then waits for L2, not for HBM.
__device__ __forceinline__ void epi_prefetch_row128(const Epilogue &e, int tok, int M, int n0, int N)
{
    if (e.residual == nullptr || tok >= M) return;
    const int cols = e.gated ? N / 2 : N, c0 = e.gated ? n0 / 2 : n0;
    const int c1 = min(c0 + (e.gated ? 64 : 128), cols);
    const __half *row = e.residual + static_cast<size_t>(tok) * cols;
    for (int c = c0; c < c1; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c1 - 1));
}

// The residual of 32 tokens and column n as epi_store_column32 wants it: before
// the sums are complete, so that its latency is not added to theirs.
__device__ __forceinline__ void epi_load_column32(const Epilogue &e, uint32_t (&rv)[16], int m0, int mrem, int n, int N)
{
    const int first = n & 1;
    if (e.residual == nullptr || n >= N) {
#pragma unroll
        for (int i = 0; i < 16; ++i) rv[i] = 0u;
    } else if (e.gated) {
        const int cols = N / 2;
        const uint16_t *r = reinterpret_cast<const uint16_t *>(e.residual) + static_cast<size_t>(m0 + first) * cols + n / 2;
#pragma unroll
        for (int i = 0; i < 16; ++i) rv[i] = 2 * i + first < mrem ? r[2 * static_cast<size_t>(i) * cols] : 0u;
    } else {
        const uint32_t *r = reinterpret_cast<const uint32_t *>(e.residual) + (static_cast<size_t>(m0 + first) * N + (n & ~1)) / 2;
#pragma unroll
        for (int i = 0; i < 16; ++i) rv[i] = 2 * i + first < mrem ? r[static_cast<size_t>(i) * N] : 0u;
    }
}

// 32 tokens m0 .. m0 + 31 (those below m0 + mrem) of column n, one column per
// lane (the accumulator layout of the tcgen05 kernels, n = n0 + lane with n0
// even); every lane of the warp calls it, lanes with n >= N write nothing.
// Gated: lanes 2j and 2j + 1 hold a gate and its column; the even lane
// finishes the even tokens and the odd lane the odd ones, one exchange per
// token pair.  rv: the residual, from epi_load_column32 (all of it was read
// before the first store: Y may be the residual's own memory).
__device__ __forceinline__ void epi_store_column32(const Epilogue &e, float (&v)[32], const uint32_t (&rv)[16],
                                                   __half *Y, int m0, int mrem, int n, int N)
{
    const bool in = n < N;
    const float b = in ? epi_bias(e, n) : 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += b;
    if (e.gated) {
        const bool odd = n & 1;
        const int cols = N / 2;
        float o[16];
        epi_with_act(e.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = __shfl_xor_sync(0xffffffffu, odd ? v[2 * i] : v[2 * i + 1], 1);
                o[i] = epi_act_of<decltype(a)::value>(odd ? x : v[2 * i]) * (odd ? v[2 * i + 1] : x);
            }
        });
        if (!in) return;
        const int first = odd ? 1 : 0;
        const size_t at = static_cast<size_t>(m0 + first) * cols + n / 2;
        const size_t step = 2 * static_cast<size_t>(cols);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] += half_lo(rv[i]);
        __half *dst = Y + at;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (2 * i + first < mrem) dst[i * step] = __float2half_rn(o[i]);
        return;
    }
    epi_with_act(e.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = epi_act_of<decltype(a)::value>(v[i]);
    });
    // the even lane of a pair finishes both its columns of the even tokens, the odd
    // lane of the odd ones: 4-byte accesses, half as many (N is even)
    const bool odd = n & 1;
    float o[32];  // of token 2 i + odd: columns n & ~1 and the next
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float x = __shfl_xor_sync(0xffffffffu, odd ? v[2 * i] : v[2 * i + 1], 1);
        o[2 * i] = odd ? x : v[2 * i];
        o[2 * i + 1] = odd ? v[2 * i + 1] : x;
    }
    if (!in) return;
    const int first = odd ? 1 : 0;
    const size_t at = (static_cast<size_t>(m0 + first) * N + (n & ~1)) / 2;  // in pairs
    uint32_t *dst = reinterpret_cast<uint32_t *>(Y) + at;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        o[2 * i] += half_lo(rv[i]);
        o[2 * i + 1] += half_hi(rv[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (2 * i + first < mrem)
            dst[static_cast<size_t>(i) * N] = pack_half2(o[2 * i], o[2 * i + 1]);
}

}  // namespace awq
