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

// One head row of D = 8 LG channels on LG neighbouring lanes: the lane's packed
// word, and on every lane the row's (step, zero point) word.
template <int LG>
__device__ __forceinline__ uint32_t quantize_row(uint4 x, uint32_t *meta, bool *nonfinite)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    __half2 mn = bits2h(w[0]), mx = mn;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mn = __hmin2(mn, bits2h(w[i]));
        mx = __hmax2(mx, bits2h(w[i]));
        bad |= (w[i] & 0x7C00u) == 0x7C00u || (w[i] & 0x7C000000u) == 0x7C000000u;
    }
    // (min x, min -x), one packed exchange per step
    __half2 e = __halves2half2(__hmin(__low2half(mn), __high2half(mn)), __hneg(__hmax(__low2half(mx), __high2half(mx))));
#pragma unroll
    for (int d = 1; d < LG; d *= 2) e = __hmin2(e, bits2h(__shfl_xor_sync(0xffffffffu, h2bits(e), d)));
    const float lo = fminf(__low2float(e), 0.0f);
    const float hi = -fminf(__high2float(e), 0.0f);
    const __half step = __float2half_rn(__fdiv_rn(fmaxf(__fsub_rn(hi, lo), 1e-5f), 15.0f));
    const float s = __half2float(step);
    const float inv = __fdiv_rn(1.0f, s);
    const float z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(bits2h(w[i]));
        const float q0 = fminf(fmaxf(rintf(__fmul_rn(f.x, inv)) + z, 0.0f), 15.0f);
        const float q1 = fminf(fmaxf(rintf(__fmul_rn(f.y, inv)) + z, 0.0f), 15.0f);
        out |= (static_cast<uint32_t>(q0) | (static_cast<uint32_t>(q1) << 4)) << (8 * i);
    }
    *meta = static_cast<uint32_t>(__half_as_ushort(step)) | (static_cast<uint32_t>(z) << 16);
    *nonfinite |= bad;
    return out;
}

// A lane group handles rows r, r + stride, ...; row = (token, head).
template <int LG>
__global__ void __launch_bounds__(kThreads) append_kernel(const StoreParams p)
{
    constexpr int D = 8 * LG;
    const int sub = static_cast<int>(threadIdx.x) % LG;
    const int64_t rows = p.T * p.c.heads;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / LG);
    bool nonfinite = false, outside = false;
    // every lane of a warp runs the same number of turns (the exchanges need all)
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / LG);
    for (int64_t r0 = first; r0 < rows; r0 += stride) {
        const int64_t r = r0 + threadIdx.x / LG;
        int64_t slot = -1;
        int head = 0;
        uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
        if (r < rows) {
            const int64_t tok = r / p.c.heads;
            head = static_cast<int>(r - tok * p.c.heads);
            slot = p.slots[tok];
            if (slot >= (p.c.num_pages << p.c.page_shift)) {
                outside = true;
                slot = -1;
            }
            if (slot >= 0) {
                kx = *reinterpret_cast<const uint4 *>(p.k + tok * p.k_stride + head * D + 8 * sub);
                vx = *reinterpret_cast<const uint4 *>(p.v + tok * p.v_stride + head * D + 8 * sub);
            }
        }
        uint32_t km, vm;
        const uint32_t kq = quantize_row<LG>(kx, &km, &nonfinite);
        const uint32_t vq = quantize_row<LG>(vx, &vm, &nonfinite);
        if (slot >= 0) {
            int row;
            uint8_t *b = block_of(p.c, slot, head, &row);
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
    const int sub = static_cast<int>(threadIdx.x) % LG;
    const int64_t rows = p.T * p.c.heads;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / LG);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / LG) + threadIdx.x / LG; r < rows; r += stride) {
        const int64_t tok = r / p.c.heads;
        const int head = static_cast<int>(r - tok * p.c.heads);
        int64_t slot = p.slots[tok];
        if (slot >= (p.c.num_pages << p.c.page_shift)) {
            report(p.status, AWQ_ERR_RANGE);
            slot = -1;
        }
        uint4 ko = make_uint4(0, 0, 0, 0), vo = ko;
        if (slot >= 0) {
            int row;
            const uint8_t *b = block_of(p.c, slot, head, &row);
            const uint32_t kq = reinterpret_cast<const uint32_t *>(b + row * (D / 2))[sub];
            const uint32_t vq = reinterpret_cast<const uint32_t *>(b + 8 * D + row * (D / 2))[sub];
            ko = dequant_word(kq, reinterpret_cast<const uint32_t *>(b + 16 * D)[row]);
            vo = dequant_word(vq, reinterpret_cast<const uint32_t *>(b + 16 * D + 64)[row]);
        }
        *reinterpret_cast<uint4 *>(p.k + r * D + 8 * sub) = ko;
        *reinterpret_cast<uint4 *>(p.v + r * D + 8 * sub) = vo;
    }
}

unsigned grid_for(int64_t rows, int lg)
{
    const int64_t per = kThreads / lg;
    const int64_t blocks = (rows + per - 1) / per;
    return static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20));
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache &c, const __half *k, int64_t k_stride, const __half *v,
                              int64_t v_stride, const int64_t *slots, int64_t T, int32_t *status, cudaStream_t st)
{
    const StoreParams prm{c, k, v, k_stride, v_stride, slots, T, status};
    if (c.D == 128)
        append_kernel<16><<<grid_for(T * c.heads, 16), kThreads, 0, st>>>(prm);
    else
        append_kernel<8><<<grid_for(T * c.heads, 8), kThreads, 0, st>>>(prm);
    return cudaGetLastError();
}

cudaError_t launch_kv4_load(const Kv4Cache &c, const int64_t *slots, int64_t T, __half *k, __half *v,
                            int32_t *status, cudaStream_t st)
{
    const LoadParams prm{c, slots, k, v, T, status};
    if (c.D == 128)
        load_kernel<16><<<grid_for(T * c.heads, 16), kThreads, 0, st>>>(prm);
    else
        load_kernel<8><<<grid_for(T * c.heads, 8), kThreads, 0, st>>>(prm);
    return cudaGetLastError();
}

}  // namespace awq
