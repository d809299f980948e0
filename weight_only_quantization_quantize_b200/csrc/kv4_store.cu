// kv4_store.cu -- keys and values of new tokens into the paged 4-bit cache,
// and back.
//
// Per token, head and tensor, over the D channels x of the head:
//   lo = min(0, min x), hi = max(0, max x)          (the grid holds zero)
//   step = binary16_RNE(max(hi - lo, 1e-5f) / 15)
//   z = clamp(rint(-lo / step), 0, 15)
//   q = clamp(rint(x * (1 / step)) + z, 0, 15)      (rint: ties to even)
// in IEEE float.  It is the weight quantizer's asymmetric grid, with two
// differences: zero is always inside the range, so that no value is clipped
// when all have one sign, and the codes use one IEEE reciprocal per group
// instead of a division per value (the quantizer runs once per layer, this on
// every token).
//
// Bound by HBM: 4 D bytes read and D + 8 written per token and head.  A group
// of D / 8 lanes holds one head row, 8 channels (16 bytes) per lane, which is
// one packed word: loads and stores are whole 16- and 4-byte words, and the
// extremes need log2(D / 8) exchanges of one packed pair (min x, min -x).
#include "kv4.cuh"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // per lane group, their loads in flight together

struct StoreParams {
    Kv4Cache c;
    const __half *k, *v;
    int64_t k_stride, v_stride;  // elements between tokens
    const int64_t *slots;
    int64_t T;
    int32_t *status;
};

__device__ __forceinline__ uint32_t h2bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits2h(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }

// Byte address of the block holding `slot` for `head`, and its row in it.
__device__ __forceinline__ uint8_t *block_of(const Kv4Cache &c, int64_t slot, int head, int *row)
{
    const int64_t page = slot >> c.page_shift;
    const int off = static_cast<int>(slot & ((1 << c.page_shift) - 1));
    *row = off & (kKvBlock - 1);
    const int64_t block = ((page * c.heads + head) << (c.page_shift - 4)) + (off >> 4);
    return c.data + block * kv4_block_bytes(c.D);
}

// (min x, min -x) of a lane's 8 channels, and through LG neighbouring lanes of
// the row; *bad becomes NaN when one is NaN or infinite.
template <int LG>
__device__ __forceinline__ __half2 row_extremes(const uint32_t (&w)[4], __half2 *bad)
{
    __half2 mn = bits2h(w[0]), mx = mn;
    const __half2 zero = __float2half2_rn(0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mn = __hmin2(mn, bits2h(w[i]));
        mx = __hmax2(mx, bits2h(w[i]));
        *bad = __hfma2(bits2h(w[i]), zero, *bad);
    }
    __half2 e = __halves2half2(__hmin(__low2half(mn), __high2half(mn)), __hneg(__hmax(__low2half(mx), __high2half(mx))));
#pragma unroll
    for (int d = 1; d < LG; d *= 2) e = __hmin2(e, bits2h(__shfl_xor_sync(0xffffffffu, h2bits(e), d)));
    return e;
}

// The grid of a row from its extremes: step and zero point as they are stored,
// and 1 / step.
__device__ __forceinline__ uint32_t row_grid(__half2 e, float *inv)
{
    const float lo = fminf(__low2float(e), 0.0f);
    const float hi = -fminf(__high2float(e), 0.0f);
    const __half step = __float2half_rn(__fdiv_rn(fmaxf(__fsub_rn(hi, lo), 1e-5f), 15.0f));
    const float s = __half2float(step);
    *inv = __frcp_rn(s);
    const float z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
    return static_cast<uint32_t>(__half_as_ushort(step)) | (static_cast<uint32_t>(z) << 16);
}

// A lane's packed word.  Adding 1.5 * 2^23 rounds a float to an integer, ties to
// even, and leaves it in the low bits: no conversion instructions, whose
// throughput would bound the kernel.
__device__ __forceinline__ uint32_t row_codes(const uint32_t (&w)[4], uint32_t meta, float inv)
{
    const int z = static_cast<int>(meta >> 16) - 0x4B400000;
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(bits2h(w[i]));
        // max(min(rounded + z, 15), 0), one instruction
        const int a = __viaddmin_s32_relu(__float_as_int(__fadd_rn(__fmul_rn(f.x, inv), 12582912.0f)), z, 15);
        const int b = __viaddmin_s32_relu(__float_as_int(__fadd_rn(__fmul_rn(f.y, inv), 12582912.0f)), z, 15);
        out += static_cast<uint32_t>(a) << (8 * i);
        out += static_cast<uint32_t>(b) << (8 * i + 4);
    }
    return out;
}

// blockIdx.y is the head; a lane group takes kTokens tokens, a block's width
// apart, whose loads are all in flight before the first is used.
template <int LG>
__global__ void __launch_bounds__(kThreads) append_kernel(const StoreParams p)
{
    constexpr int D = 8 * LG;
    constexpr int kGroups = kThreads / LG;
    const int sub = static_cast<int>(threadIdx.x) % LG, head = static_cast<int>(blockIdx.y);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kGroups * kTokens) + threadIdx.x / LG;
    const int64_t end = p.c.num_pages << p.c.page_shift;
    bool nonfinite = false, outside = false;
    int64_t slot[kTokens];
    uint4 kx[kTokens], vx[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int64_t tok = first + i * kGroups;
        slot[i] = -1;
        kx[i] = vx[i] = make_uint4(0, 0, 0, 0);
        if (tok < p.T) {
            slot[i] = p.slots[tok];
            kx[i] = *reinterpret_cast<const uint4 *>(p.k + tok * p.k_stride + head * D + 8 * sub);
            vx[i] = *reinterpret_cast<const uint4 *>(p.v + tok * p.v_stride + head * D + 8 * sub);
        }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        if (slot[i] >= end) {
            outside = true;
            slot[i] = -1;
        }
        // every lane takes part in the exchanges; a row that is not stored is not judged either
        const uint32_t kw[4] = {kx[i].x, kx[i].y, kx[i].z, kx[i].w}, vw[4] = {vx[i].x, vx[i].y, vx[i].z, vx[i].w};
        __half2 bad2 = __float2half2_rn(0.0f);
        const __half2 ke = row_extremes<LG>(kw, &bad2), ve = row_extremes<LG>(vw, &bad2);
        // half of the lanes work out the key's grid, half the value's
        float inv;
        const uint32_t meta = row_grid(sub < LG / 2 ? ke : ve, &inv);
        const uint32_t km = __shfl_sync(0xffffffffu, meta, 0, LG), vm = __shfl_sync(0xffffffffu, meta, LG / 2, LG);
        const float ki = __shfl_sync(0xffffffffu, inv, 0, LG), vi = __shfl_sync(0xffffffffu, inv, LG / 2, LG);
        const uint32_t kq = row_codes(kw, km, ki), vq = row_codes(vw, vm, vi);
        const bool bad = __hisnan(__low2half(bad2)) || __hisnan(__high2half(bad2));
        if (slot[i] >= 0) {
            nonfinite |= bad;
            int row;
            uint8_t *b = block_of(p.c, slot[i], head, &row);
            reinterpret_cast<uint32_t *>(b + row * (D / 2))[sub] = kq;
            reinterpret_cast<uint32_t *>(b + 8 * D + row * (D / 2))[sub] = vq;
            if (sub < 2) reinterpret_cast<uint32_t *>(b + 16 * D + 64 * sub)[row] = sub ? vm : km;
        }
    }
    if (outside) report(p.status, AWQ_ERR_RANGE);
    if (nonfinite) report(p.status, AWQ_ERR_NONFINITE);
}

struct LoadParams {
    Kv4Cache c;
    const int64_t *slots;
    __half *k, *v;
    int64_t T;
    int32_t *status;
};

// (q - z) * step of one packed word, 8 channels, each rounded once to binary16
// ((q - z) is exact in binary16).
__device__ __forceinline__ uint4 dequant_word(uint32_t w, uint32_t meta)
{
    const int z = static_cast<int>(meta >> 16);
    const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(meta)));
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = static_cast<float>(static_cast<int>((w >> (8 * i)) & 15u) - z) * s;
        const float b = static_cast<float>(static_cast<int>((w >> (8 * i + 4)) & 15u) - z) * s;
        o[i] = h2bits(__floats2half2_rn(a, b));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int LG>
__global__ void __launch_bounds__(kThreads) load_kernel(const LoadParams p)
{
    constexpr int D = 8 * LG;
    constexpr int kGroups = kThreads / LG;
    const int sub = static_cast<int>(threadIdx.x) % LG, head = static_cast<int>(blockIdx.y);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kGroups * kTokens) + threadIdx.x / LG;
    const int64_t end = p.c.num_pages << p.c.page_shift;
    int64_t slot[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int64_t tok = first + i * kGroups;
        slot[i] = tok < p.T ? p.slots[tok] : -1;
        if (slot[i] >= end) {
            report(p.status, AWQ_ERR_RANGE);
            slot[i] = -1;
        }
    }
    uint32_t kq[kTokens], vq[kTokens], km[kTokens], vm[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        kq[i] = vq[i] = km[i] = vm[i] = 0;  // reads as zeros
        if (slot[i] >= 0) {
            int row;
            const uint8_t *b = block_of(p.c, slot[i], head, &row);
            kq[i] = reinterpret_cast<const uint32_t *>(b + row * (D / 2))[sub];
            vq[i] = reinterpret_cast<const uint32_t *>(b + 8 * D + row * (D / 2))[sub];
            km[i] = reinterpret_cast<const uint32_t *>(b + 16 * D)[row];
            vm[i] = reinterpret_cast<const uint32_t *>(b + 16 * D + 64)[row];
        }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int64_t tok = first + i * kGroups;
        if (tok >= p.T) break;
        const int64_t r = tok * p.c.heads + head;
        *reinterpret_cast<uint4 *>(p.k + r * D + 8 * sub) = dequant_word(kq[i], km[i]);
        *reinterpret_cast<uint4 *>(p.v + r * D + 8 * sub) = dequant_word(vq[i], vm[i]);
    }
}

dim3 grid_for(int64_t T, int heads, int lg)
{
    const int64_t per = static_cast<int64_t>(kThreads / lg) * kTokens;
    return dim3(static_cast<unsigned>((T + per - 1) / per), static_cast<unsigned>(heads));
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache &c, const __half *k, int64_t k_stride, const __half *v,
                              int64_t v_stride, const int64_t *slots, int64_t T, int32_t *status, cudaStream_t st)
{
    const StoreParams prm{c, k, v, k_stride, v_stride, slots, T, status};
    if (c.D == 128)
        append_kernel<16><<<grid_for(T, c.heads, 16), kThreads, 0, st>>>(prm);
    else
        append_kernel<8><<<grid_for(T, c.heads, 8), kThreads, 0, st>>>(prm);
    return cudaGetLastError();
}

cudaError_t launch_kv4_load(const Kv4Cache &c, const int64_t *slots, int64_t T, __half *k, __half *v,
                            int32_t *status, cudaStream_t st)
{
    const LoadParams prm{c, slots, k, v, T, status};
    if (c.D == 128)
        load_kernel<16><<<grid_for(T, c.heads, 16), kThreads, 0, st>>>(prm);
    else
        load_kernel<8><<<grid_for(T, c.heads, 8), kThreads, 0, st>>>(prm);
    return cudaGetLastError();
}

}  // namespace awq
