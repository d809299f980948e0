// kv4_attend.cu -- attention over the paged 4-bit key/value cache for few query
// rows per key/value head (single tokens and short runs of tokens): the
// HBM-bound regime, every cached code read once.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - max_j)
//   k_j = step_j (c_j - z_j), and v_j likewise, with integer codes c, so
//   q_i . k_j   = step_j (q_i . (c_j - z_j))
//   sum_j p v_j = sum_j (p_ij step_j) (c_j - z_j)
// The steps stay out of the products, whose operands c - z are exact in
// binary16: the tensor cores (mma.sync m16n8k16, tokens or channels as rows,
// query rows as the 8 columns) multiply integers, and the float accumulators
// hold no offset that would have to cancel.  (Feeding the masked nibbles as
// binary16 subnormals, without any unpacking arithmetic, was built first and
// measured to lose 6 to 10 bits of the sum.)  The unpack is one AND-OR per pair of codes into the
// mantissa of 1024 and one packed add or multiply-add that takes 1024 (or 64)
// and z off; integer and FMA pipes share it.  A value needs the same channel
// of two tokens in one register: one byte permute per pair of words gives that.
//
// Roundings: p_ij step_j to binary16 for the second product (the row sum uses
// the unrounded float p), and the output.  The reference of the
// exponentials is kept on s + log2(step of v), and 2^8 above the largest
// weight, so that the weights neither overflow (below 2^14 between two
// updates) nor lose bits to subnormals within 2^-22 of the largest one.
//
// Work split: the (request, row block, head) items of all requests form one
// line of 64-token tiles, and every CTA takes an equal run of it, whatever the
// lengths.  Runs that cut an item leave (max, sum, numerator) in the workspace
// and a second kernel joins them in a fixed order: no atomics, no waiting
// between CTAs, the same bits every time.
//
// A CTA is four independent warps with a ring of kStages tiles each, filled by
// bulk copies that the warp's lanes issue in turn: a block of 16 tokens (keys,
// values, steps, zero points) is one contiguous piece of the page.
#include <type_traits>

#include "awq_kernels.cuh"
#include "kv4.cuh"

namespace awq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 64;       // tokens per ring stage
constexpr int kTileBlocks = kTile / kKvBlock;
// An item's start and end (queries in, joins of warps, output) in tiles: the
// runs are equal in this measure.  48 ragged requests of 819..16384 tokens, 8
// heads: 132 us at 0, 126 at 2, 117 at 4, 113 at 6 to 12.
constexpr int kItemCost = 8;
constexpr int kMaxCtas = 640;
constexpr int kMinTiles = 4;    // tiles per CTA at least, one per warp
constexpr float kGain = 8.0f;   // log2 of the largest weight after an update
constexpr float kSlack = 13.0f; // log2 of the weight, without its step's fraction, that forces one
constexpr float kLimit = 16384.0f;  // weights above 2^(kSlack + 1) ask for it
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NT>
struct Cfg {
    static constexpr int kRows = 8 * NT;
    static constexpr int kStages = 2;
    static constexpr int kBlock = kv4_block_bytes(D);
    static constexpr int kStage = kTileBlocks * kBlock;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kMerge = 4 * 32 * (NT * (D / 16) * 4 + 4 * NT);  // floats of one warp
    static constexpr int kBars = 8 * kWarps * kStages;
    static constexpr size_t kSmem = 128 + kRing + kMerge + kBars + 4 * kWarps * kStages + 64;
    static constexpr int kCtasPerSm = NT == 1 ? 3 : 2;
};

// What the joining kernel has to know of an item that a CTA begins and others go on with.
struct Desc {
    int count;      // CTAs that hold a part of it; 0: none
    int first_row;  // its first row among the request's (queries times heads of the group)
    int rows;       // of the request
    int head, q0, pad[3];
};

struct Params {
    Kv4AttendArgs a;
    Desc *desc;      // [grid]
    float2 *ml;      // [2 grid][rows]: (reference, sum) of a part
    float *part;     // [2 grid][rows][D]
    int group;
    int64_t max_rows;  // requests with more rows are another kernel's
    UnpackConsts uk;
};

struct Request {
    int len, nq, q0;   // cached tokens, queries, first query row
    int lo;            // the first position that any query sees
    int tile0, tiles;  // first tile that any query reads, tiles from there
    int items;         // row blocks times heads
    int units;         // of one item: its tiles, and kItemCost for what it costs besides
};

template <int ROWS>
__device__ __forceinline__ Request request_at(const Params &p, int b)
{
    const Kv4AttendArgs &a = p.a;
    Request r;
    const long long most = static_cast<long long>(a.tab.max_pages) << a.cache.page_shift;
    r.len = a.tab.lens[b];
    r.q0 = a.tab.cu ? a.tab.cu[b] : b;
    const long long q1 = a.tab.cu ? a.tab.cu[b + 1] : b + 1;
    bool bad = false;
    if (r.len < 0 || r.len > most) {
        bad = true;
        r.len = r.len < 0 ? 0 : static_cast<int>(most);
    }
    long long nq = q1 - r.q0;
    if (r.q0 < 0 || nq < 0 || q1 > a.T || nq > a.max_new) {
        bad = true;
        nq = 0;
    }
    if (bad) report(a.status, AWQ_ERR_RANGE);
    r.nq = static_cast<int>(nq);
    const long long first = a.window > 0 ? static_cast<long long>(r.len) - r.nq - a.window + 1 : 0;
    r.lo = first > 0 ? static_cast<int>(first) : 0;
    r.tile0 = r.lo / kTile;
    const int t = (r.len + kTile - 1) / kTile - r.tile0;
    r.tiles = t < 1 ? 1 : t;  // rows that see nothing are still written
    r.items = static_cast<int64_t>(r.nq) * p.group > p.max_rows ? 0 : (r.nq * p.group + ROWS - 1) / ROWS * a.cache.heads;
    r.units = r.tiles + kItemCost;
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Plain loads, so that the compiler may move them between the waits.
__device__ __forceinline__ uint32_t word_at(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }

template <int W>
__device__ __forceinline__ void words_at(const uint8_t *p, uint32_t (&w)[W])
{
    if constexpr (W == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (W == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x; w[1] = x.y;
    } else {
        w[0] = word_at(p);
    }
}

// D = A * B
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// (step, zero point) word of a token
__device__ __forceinline__ float meta_step(uint32_t m) { return __half2float(__ushort_as_half(static_cast<uint16_t>(m))); }
// -(1024 + z) of two tokens' words (of one token: twice the same word), packed
// in this order, or swapped with the other selector
constexpr uint32_t kInOrder = 0x7632, kSwapped = 0x3276;
__device__ __forceinline__ uint32_t meta_zeros(uint32_t m0, uint32_t m1, uint32_t order)
{
    return (__byte_perm(m0, m1, order) & 0x000F000Fu) | 0xE400E400u;  // finite, whatever the word holds
}

// Codes of a word's nibbles 0 and 4 (low) or 1 and 5 (high), as they lie in
// both halves, minus zero points: za = -(1024 + z), zb = -(64 + z).
__device__ __forceinline__ uint32_t codes_low(uint32_t w, uint32_t za, const UnpackConsts &k)
{
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"((w & k.mask_lo) | k.magic), "r"(za));
    return d;
}

__device__ __forceinline__ uint32_t codes_high(uint32_t w, uint32_t zb, const UnpackConsts &k)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"((w & k.mask_hi) | k.magic), "r"(k.sixteenth), "r"(zb));
    return d;
}

__device__ __forceinline__ uint32_t zeros_high(uint32_t za)  // -(1024 + z) + 960
{
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(za), "r"(0x63806380u));
    return d;
}
// floor(log2(step)), and -14 for subnormal steps: step < 2^(this + 1)
__device__ __forceinline__ float meta_exp(uint32_t m)
{
    const int e = (m >> 10) & 31;
    return static_cast<float>((e < 1 ? 1 : e) - 15);
}

// The block row that row r (0..7) of the first product stands for.  The second
// product reads rows 2 t and 2 t + 1 for t = 0..3 together: this order puts
// two even and two odd rows in each set, which halves the bank conflicts of
// rows 64 bytes long, and keeps rows 2 i and 2 i + 1 of opposite parity.
__device__ __forceinline__ int token_of(int r) { return r ^ ((r >> 1) & 1); }

template <int D, int NT>
struct Warp {
    float o[NT][D / 16][4];     // numerators: [column tile][MMA][row/column]
    float m[NT][2], l[NT][2];
    uint32_t q[NT][D / 32][2][2];  // the second operand of the first product
    int hi[NT][2], lo[NT][2];   // keys lo < j <= hi of the lane's two rows
};

template <int D, int NT>
__device__ __forceinline__ void start_item(Warp<D, NT> &w, const Params &p, const Request &r, int item, int lane)
{
    constexpr int ROWS = 8 * NT;
    const int gid = lane >> 2, t = lane & 3;
    const int rb = item / p.a.cache.heads, head = item - rb * p.a.cache.heads;
    const int rows = r.nq * p.group;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) w.o[n][i][c] = 0.0f;
        const int row = rb * ROWS + 8 * n + gid;
        const bool in = row < rows;
        const int i = in ? row / p.group : 0;
        const __half *src = p.a.q + (r.q0 + i) * p.a.q_stride +
                            static_cast<int64_t>(head * p.group + (in ? row - i * p.group : 0)) * D + 8 * (D / 32) * t;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            const uint4 x = in ? __ldg(reinterpret_cast<const uint4 *>(src + 8 * k)) : make_uint4(0, 0, 0, 0);
            // channels (0,4), (2,6) against the low nibbles, (1,5), (3,7) against the high ones
            w.q[n][k][0][0] = __byte_perm(x.x, x.z, 0x5410);
            w.q[n][k][0][1] = __byte_perm(x.y, x.w, 0x5410);
            w.q[n][k][1][0] = __byte_perm(x.x, x.z, 0x7632);
            w.q[n][k][1][1] = __byte_perm(x.y, x.w, 0x7632);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            w.l[n][c] = 0.0f;
            const int own = rb * ROWS + 8 * n + 2 * t + c;
            const int pos = max(r.len - r.nq + own / p.group, -1);  // -1: before the first token
            w.hi[n][c] = own < rows ? pos : -1;
            w.m[n][c] = own < rows ? -INFINITY : 0.0f;  // rows that stand for nothing are never written
            w.lo[n][c] = p.a.window > 0 ? pos - p.a.window : -1;
        }
    }
}

// Two blocks, 32 tokens tok .. tok + 31.  full: every token is seen by every
// row, and every row has a reference; otherwise rows are masked and blocks
// whose bit in `have` is clear hold nothing.  NT of the warp's WT column tiles
// hold rows.
template <int D, int WT, int NT>
__device__ __forceinline__ void tile_step(Warp<D, WT> &w, const uint8_t *stage, int tok, bool full, int have, float c1,
                                          const UnpackConsts &uk, int lane)
{
    constexpr int KW = D / 32;  // key words per lane and row
    constexpr int VW = D / 64;  // value words per lane and token
    constexpr int RB = D / 2;   // bytes of a row
    const int gid = lane >> 2, t = lane & 3;
    const int ra = token_of(gid);
    float s[2][NT][4], f[2][2];  // products of q and codes; what a token's step and the scale make of them
    uint32_t vm[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint8_t *base = stage + b * kv4_block_bytes(D);
        uint32_t ka[KW], kb[KW];
        words_at<KW>(base + ra * RB + t * (4 * KW), ka);
        words_at<KW>(base + (ra + 8) * RB + t * (4 * KW), kb);
        const uint32_t ma = word_at(base + 16 * D + 4 * ra), mb = word_at(base + 16 * D + 4 * (ra + 8));
        vm[b][0] = word_at(base + 16 * D + 64 + 4 * ra);
        vm[b][1] = word_at(base + 16 * D + 64 + 4 * (ra + 8));
        const uint32_t za = meta_zeros(ma, ma, kInOrder), zb = meta_zeros(mb, mb, kInOrder), ya = zeros_high(za), yb = zeros_high(zb);
        float al[NT][4], ah[NT][4];
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            const uint32_t a8 = ka[k] >> 8, b8 = kb[k] >> 8;
            const uint32_t lo[4] = {codes_low(ka[k], za, uk), codes_low(kb[k], zb, uk), codes_low(a8, za, uk), codes_low(b8, zb, uk)};
            const uint32_t hi[4] = {codes_high(ka[k], ya, uk), codes_high(kb[k], yb, uk), codes_high(a8, ya, uk), codes_high(b8, yb, uk)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (k == 0) {
                    mma_first(al[n], lo, w.q[n][k][0][0], w.q[n][k][0][1]);
                    mma_first(ah[n], hi, w.q[n][k][1][0], w.q[n][k][1][1]);
                } else {
                    mma_16816(al[n], lo, w.q[n][k][0][0], w.q[n][k][0][1]);
                    mma_16816(ah[n], hi, w.q[n][k][1][0], w.q[n][k][1][1]);
                }
            }
        }
        f[b][0] = meta_step(ma) * c1;
        f[b][1] = meta_step(mb) * c1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[b][n][c] = al[n][c] + ah[n][c];
    }
    // Weights with the reference as it stands.  It is moved, one vote per tile,
    // only when a weight passes 2^(kSlack + 1).
    uint32_t pk[2][NT][2];
    float sum[NT][2];
    bool over = !full;
    if (full) {
        __half2 big = __float2half2_rn(0.0f);
#pragma unroll
        for (int n = 0; n < NT; ++n) sum[n][0] = sum[n][1] = 0.0f;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float step = meta_step(vm[b][h]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float e0 = ex2(fmaf(f[b][h], s[b][n][2 * h], -w.m[n][0]));
                    const float e1 = ex2(fmaf(f[b][h], s[b][n][2 * h + 1], -w.m[n][1]));
                    sum[n][0] += e0;
                    sum[n][1] += e1;
                    pk[b][n][h] = pack2(e0 * step, e1 * step);
                    big = __hmax2(big, *reinterpret_cast<__half2 *>(&pk[b][n][h]));
                }
            }
        over = !__hble2(big, __float2half2_rn(kLimit));
    }
    if (__any_sync(0xffffffffu, over)) {
        // floor(log2(step)) of each value joins the logits: weights include their steps
        float ev[2][2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ev[b][h] = meta_exp(vm[b][h]);
                const int j = tok + 16 * b + 8 * h + ra;
                const bool there = (have >> b) & 1;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // select, never multiply: what a masked place holds may be anything; a
                        // product that is not finite (x - x is then NaN) is not taken for one
                        const bool seen = full || (there && j <= w.hi[n][c] && j > w.lo[n][c]);
                        const float x = s[b][n][2 * h + c];
                        s[b][n][2 * h + c] = seen ? fmaf(f[b][h], x, x - x) : -INFINITY;
                    }
            }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = fmaxf(fmaxf(s[0][n][c] + ev[0][0], s[0][n][2 + c] + ev[0][1]),
                                fmaxf(s[1][n][c] + ev[1][0], s[1][n][2 + c] + ev[1][1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                if (x > w.m[n][c] + kSlack) {
                    const float next = x - kGain;
                    const float g = ex2(w.m[n][c] - next);  // 0 for the first one
                    w.m[n][c] = next;
                    w.l[n][c] *= g;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        w.o[n][i][c] *= g;
                        w.o[n][i][2 + c] *= g;
                    }
                }
                sum[n][c] = 0.0f;
            }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float step = meta_step(vm[b][h]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float pv[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float x = s[b][n][2 * h + c];
                        const float e = x == -INFINITY ? 0.0f : ex2(x - w.m[n][c]);
                        sum[n][c] += e;
                        pv[c] = x == -INFINITY ? 0.0f : e * step;
                    }
                    pk[b][n][h] = pack2(pv[0], pv[1]);
                }
            }
    }
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        w.l[n][0] += sum[n][0];
        w.l[n][1] += sum[n][1];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) pb[b][n][h] = transpose8x8(pk[b][n][h]);
    }
    const int t0 = token_of(2 * t), t1 = token_of(2 * t + 1);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint8_t *base = stage + b * kv4_block_bytes(D) + 8 * D + gid * (4 * VW);
        const uint8_t *meta = stage + b * kv4_block_bytes(D) + 16 * D + 64;
        uint32_t m0[2], m1[2];  // rows 2 t and 2 t + 1, t0 and t1 in some order, and those 8 on
        words_at<2>(meta + 8 * t, m0);
        words_at<2>(meta + 8 * t + 32, m1);
        const uint32_t order = (t & 1) ? kSwapped : kInOrder;
        const uint32_t z0 = meta_zeros(m0[0], m0[1], order), z1 = meta_zeros(m1[0], m1[1], order);
        const uint32_t y0 = zeros_high(z0), y1 = zeros_high(z1);
        uint32_t v0[VW], v1[VW], v2[VW], v3[VW];
        words_at<VW>(base + t0 * RB, v0);
        words_at<VW>(base + t1 * RB, v1);
        words_at<VW>(base + (t0 + 8) * RB, v2);
        words_at<VW>(base + (t1 + 8) * RB, v3);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            const uint32_t u[4] = {__byte_perm(v0[i], v1[i], 0x5410), __byte_perm(v0[i], v1[i], 0x7632),
                                   __byte_perm(v2[i], v3[i], 0x5410), __byte_perm(v2[i], v3[i], 0x7632)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int sh = (j & 2) ? 8 : 0;
                uint32_t a[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    a[e] = (j & 1) ? codes_high(u[e] >> sh, e < 2 ? y0 : y1, uk)
                                     : codes_low(u[e] >> sh, e < 2 ? z0 : z1, uk);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_16816(w.o[n][4 * i + j], a, pb[b][n][0], pb[b][n][1]);
            }
        }
    }
}

// Joins another part of the same rows into (m, l, o).
__device__ __forceinline__ void join_weights(float &m, float m2, float &f, float &f2)
{
    const float top = fmaxf(m, m2);
    f = m == -INFINITY ? 0.0f : ex2(m - top);
    f2 = m2 == -INFINITY ? 0.0f : ex2(m2 - top);
    m = top;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtasPerSm) attend_kernel(const Params p)
{
    using C = Cfg<D, NT>;
    extern __shared__ uint8_t smem_dyn[];
    __shared__ uint32_t s_sum[kWarps];
    __shared__ int s_b;
    __shared__ uint32_t s_rem;
    const uint32_t raw = smem_u32(smem_dyn);
    uint8_t *smem = smem_dyn + ((128u - (raw & 127u)) & 127u);
    float *merge = reinterpret_cast<float *>(smem + C::kRing);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kRing + C::kMerge);
    int *haves = reinterpret_cast<int *>(smem + C::kRing + C::kMerge + C::kBars);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = static_cast<int>(blockIdx.x);
    const Kv4AttendArgs &a = p.a;
    const int heads = a.cache.heads;
    pdl_launch_dependents();

    // ---------------------------------------------------------------- this CTA's run of tiles
    if (threadIdx.x < kWarps * C::kStages) mbar_init(&bars[threadIdx.x], 1);
    fence_barrier_init();
    const int per = (a.tab.B + kThreads - 1) / kThreads;
    const int bfirst = static_cast<int>(threadIdx.x) * per;
    uint32_t mine = 0;
    for (int j = 0; j < per && bfirst + j < a.tab.B; ++j) {
        const Request r = request_at<C::kRows>(p, bfirst + j);
        mine += static_cast<uint32_t>(r.items) * r.units;
    }
    uint32_t pre = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, pre, d);
        if (lane >= d) pre += y;
    }
    if (lane == 31) s_sum[warp] = pre;
    __syncthreads();
    uint32_t U = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) pre += s_sum[i];
        U += s_sum[i];
    }
    pre -= mine;
    uint32_t G = U / kMinTiles;
    G = G < 1 ? 1 : G > gridDim.x ? gridDim.x : G;
    const uint32_t share = U / G, rest = U % G;
    auto begin_of = [&](uint32_t c) { return c * share + (c < rest ? c : rest); };
    const uint32_t c = static_cast<uint32_t>(cta);
    const uint32_t u0 = c < G ? begin_of(c) : U, u1 = c < G ? begin_of(c + 1) : U;
    if (u0 >= u1) {
        if (threadIdx.x == 0) p.desc[cta].count = 0;
        return;
    }
    if (u0 >= pre && u0 < pre + mine) {
        uint32_t rem = u0 - pre;
        int b = bfirst;
        for (; b + 1 < a.tab.B; ++b) {
            const Request r = request_at<C::kRows>(p, b);
            const uint32_t n = static_cast<uint32_t>(r.items) * r.units;
            if (rem < n) break;
            rem -= n;
        }
        s_b = b;
        s_rem = rem;
    }
    __syncthreads();

    // ---------------------------------------------------------------- the warp's loads
    const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStage);
    uint64_t *bar = bars + warp * C::kStages;
    const uint32_t bar0 = smem_u32(bar);
    int *have_of = haves + warp * C::kStages;
    // load cursor: request, item, first tile of the segment (within the item),
    // the segment's tiles, the next one for this warp
    int lb = s_b;
    Request lr = request_at<C::kRows>(p, lb);
    int litem = static_cast<int>(s_rem / lr.units);
    // the segment [v, v + n) of an item's units: tiles from max(v - kItemCost, 0)
    int lv = static_cast<int>(s_rem % lr.units);
    uint32_t ln = min(static_cast<uint32_t>(lr.units - lv), u1 - u0);
    int lt0 = max(lv - kItemCost, 0);
    uint32_t lu = u0;
    int lseg = max(lv + static_cast<int>(ln) - kItemCost, 0) - lt0;
    int lnext = warp;
    // the blocks of 8 of the warp's tiles, one block per lane: lane 4 i + j copies
    // `bytes` bytes of tile i (its blocks from j on, up to the next copy)
    const uint8_t *src = nullptr;
    uint32_t bytes = 0, expect = 0;
    int held = 0;         // bits of the tile's blocks that are there
    int turn = 8;         // the tile of the batch that is next
    int issued = 0;       // tiles asked for; the ring slot of the next one
    int ist = 0;

    auto issue = [&]() {
        while (lnext >= lseg) {  // on to the next segment
            lu += ln;
            ln = 0;
            if (lu >= u1) {
                lseg = lnext = 0;
                return;
            }
            lt0 = 0;
            if (++litem >= lr.items && lb + 1 < a.tab.B) {
                litem = 0;
                do lr = request_at<C::kRows>(p, ++lb);
                while (lr.items == 0 && lb + 1 < a.tab.B);
            }
            ln = min(static_cast<uint32_t>(lr.units), u1 - lu);
            lseg = max(static_cast<int>(ln) - kItemCost, 0);
            lnext = warp;
            turn = 8;
        }
        if (turn == 8) {
            turn = 0;
            const int tl = lnext + kWarps * (lane >> 2), j = lane & 3;
            const int tok = (lr.tile0 + lt0 + tl) * kTile + kKvBlock * j;
            const int sh = a.cache.page_shift - 4;
            bool there = false;
            // blocks before the first position that any query sees may have lost their pages
            if (tl < lseg && tok < lr.len && tok + kKvBlock > lr.lo) {
                const int page = a.tab.block_table[static_cast<size_t>(lb) * a.tab.max_pages + (tok >> a.cache.page_shift)];
                there = page >= 0 && page < a.cache.num_pages;
                if (!there) report(a.status, AWQ_ERR_RANGE);
                const int64_t at = (tok >> 4) & ((1 << sh) - 1);
                src = a.cache.data + (((static_cast<int64_t>(page) * heads + litem % heads) << sh) + at) * C::kBlock;
            }
            held = (__ballot_sync(0xffffffffu, there) >> (lane & 28)) & 15;
            expect = __popc(held) * C::kBlock;
            // the blocks of one page that are there lie together: the first one's lane copies them all
            const int size = sh > 2 ? 4 : 1 << sh, begin = j & ~(size - 1);
            const bool lead = there && (j == begin || !((held >> (j - 1)) & 1));
            bytes = lead ? __popc((held >> j) & ((1 << (begin + size - j)) - 1)) * C::kBlock : 0;
        }
        if ((lane >> 2) == turn) {
            const uint32_t mb = bar0 + 8 * ist;
            if ((lane & 3) == 0) {
                mbar_arrive_expect_tx(&bar[ist], expect);
                have_of[ist] = held;
            }
            __syncwarp(15u << (4 * turn));  // the barrier expects the bytes before they can arrive
            if (bytes) bulk_load(ring + ist * C::kStage + (lane & 3) * C::kBlock, src, bytes, mb);
        }
        ++turn;
        ++issued;
        if (++ist == C::kStages) ist = 0;
        lnext += kWarps;
    };
    for (int i = 0; i < C::kStages; ++i) issue();
    __syncwarp();

    // ---------------------------------------------------------------- segments
    int b = s_b;
    Request r = request_at<C::kRows>(p, b);
    int item = static_cast<int>(s_rem / r.units);
    int v = static_cast<int>(s_rem % r.units);
    uint32_t u = u0;
    int st = 0;         // ring slot of the next tile and the parity of its use
    uint32_t ph = 0;
    bool dead = false;
    bool split_tail = false;
    const float c1 = a.scale * kLog2e;
    Warp<D, NT> w;
    while (u < u1) {
        const int n = static_cast<int>(min(static_cast<uint32_t>(r.units - v), u1 - u));
        const int t0 = max(v - kItemCost, 0);
        const int seg = max(v + n - kItemCost, 0) - t0;
        if (warp < seg) {
            start_item<D, NT>(w, p, r, item, lane);
            const int rb = item / heads;
            const bool wide = r.nq * p.group - rb * C::kRows > 8;
            const int ifirst = rb * C::kRows / p.group;
            const int ilast = min((rb * C::kRows + C::kRows - 1) / p.group, r.nq - 1);
            const int pfirst = r.len - r.nq + ifirst;                       // the earliest row's position
            const int wlast = a.window > 0 ? max(r.len - r.nq + ilast, -1) - a.window : -1;
            // tiles first .. last - 1 of the segment hold only tokens that every row sees
            const int base = r.tile0 + t0;
            const int first = (wlast + kTile) / kTile - base;  // the first tile that begins above wlast
            const int last = min(r.len, pfirst + 1) / kTile - base;
            bool ready = false;  // every row has a reference
            for (int k = warp; k < seg; k += kWarps) {
                if (!dead && !__all_sync(0xffffffffu, mbar_wait(&bar[st], ph))) {
                    dead = true;
                    if (lane == 0) report(a.status, AWQ_ERR_DEVICE_TIMEOUT);
                }
                const uint8_t *stage = smem + warp * (C::kStages * C::kStage) + st * C::kStage;
                const int have = have_of[st];
                // the second column tile may hold no rows (single tokens among longer runs)
                auto blocks = [&](auto tiles, bool full) {
                    constexpr int A = decltype(tiles)::value;
                    if (full) {
#pragma unroll
                        for (int b = 0; b < kTileBlocks; b += 2)
                            tile_step<D, NT, A>(w, stage + b * C::kBlock, 0, true, 3, c1, p.uk, lane);
                    } else {
                        for (int b = 0; b < kTileBlocks; b += 2)
                            if ((have >> b) & 3)
                                tile_step<D, NT, A>(w, stage + b * C::kBlock, (base + k) * kTile + b * kKvBlock, false,
                                                    (have >> b) & 3, c1, p.uk, lane);
                    }
                };
                const bool full = ready && have == (1 << kTileBlocks) - 1 && k >= first && k < last;
                if (NT == 1 || wide)
                    blocks(std::integral_constant<int, NT>{}, full);
                else
                    blocks(std::integral_constant<int, 1>{}, full);
                if (!full) {
                    bool set = true;
#pragma unroll
                    for (int n = 0; n < NT; ++n) set = set && w.m[n][0] != -INFINITY && w.m[n][1] != -INFINITY;
                    ready = __all_sync(0xffffffffu, set);
                }
                if (++st == C::kStages) {
                    st = 0;
                    ph ^= 1u;
                }
                __syncwarp();
                if (!dead) issue();
                __syncwarp();
            }
            // the lanes' sums over tokens
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) w.l[n][cc] += __shfl_xor_sync(0xffffffffu, w.l[n][cc], d);
                }
        }
        // the warps' parts, last warp first, into the first warp
        const int parts = seg < kWarps ? seg : kWarps;
        for (int src = parts - 1; src >= 0; --src) {
            if (warp == src) {
                if (src < parts - 1) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int cc = 0; cc < 2; ++cc) {
                            const float m2 = merge[(4 * n + 2 * cc) * 32 + lane], l2 = merge[(4 * n + 2 * cc + 1) * 32 + lane];
                            float f, f2;
                            join_weights(w.m[n][cc], m2, f, f2);
                            w.l[n][cc] = w.l[n][cc] * f + l2 * f2;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const float o2 = merge[(4 * NT + (n * (D / 16) + i) * 4 + 2 * h + cc) * 32 + lane];
                                    w.o[n][i][2 * h + cc] = w.o[n][i][2 * h + cc] * f + o2 * f2;
                                }
                        }
                }
                if (src > 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int cc = 0; cc < 2; ++cc) {
                            merge[(4 * n + 2 * cc) * 32 + lane] = w.m[n][cc];
                            merge[(4 * n + 2 * cc + 1) * 32 + lane] = w.l[n][cc];
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    merge[(4 * NT + (n * (D / 16) + i) * 4 + 2 * h + cc) * 32 + lane] = w.o[n][i][2 * h + cc];
                        }
                }
            }
            if (parts > 1) __syncthreads();
        }
        const bool whole = seg == r.tiles;
        if (warp == 0 && seg > 0) {
            const int gid = lane >> 2, t = lane & 3;
            const int rb = item / heads, head = item - rb * heads;
            const size_t slot = (2 * static_cast<size_t>(cta) + (t0 == 0 ? 1 : 0)) * C::kRows;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    const int col = 8 * n + 2 * t + cc;
                    const int row = rb * C::kRows + col;
                    if (row >= r.nq * p.group) continue;
                    if (whole) {
                        const float inv = w.l[n][cc] > 0.0f ? 1.0f / w.l[n][cc] : 0.0f;
                        const int i = row / p.group;
                        __half *dst = a.out + (static_cast<int64_t>(r.q0 + i) * a.q_heads + head * p.group + row - i * p.group) * D +
                                      gid * (D / 8);
#pragma unroll
                        for (int v = 0; v < D / 64; ++v) {
                            const float *lo = &w.o[n][4 * v][0];
                            uint4 x;
                            x.x = pack2(lo[cc] * inv, lo[4 + cc] * inv);
                            x.y = pack2(lo[8 + cc] * inv, lo[12 + cc] * inv);
                            x.z = pack2(lo[2 + cc] * inv, lo[6 + cc] * inv);
                            x.w = pack2(lo[10 + cc] * inv, lo[14 + cc] * inv);
                            reinterpret_cast<uint4 *>(dst)[v] = x;
                        }
                    } else {
                        if (gid == 0) p.ml[slot + col] = make_float2(w.m[n][cc], w.l[n][cc]);
                        float *dst = p.part + (slot + col) * D + gid * (D / 8);
#pragma unroll
                        for (int v = 0; v < D / 64; ++v) {
                            const float *lo = &w.o[n][4 * v][0];
                            reinterpret_cast<float4 *>(dst)[2 * v] = make_float4(lo[cc], lo[4 + cc], lo[8 + cc], lo[12 + cc]);
                            reinterpret_cast<float4 *>(dst)[2 * v + 1] = make_float4(lo[2 + cc], lo[6 + cc], lo[10 + cc], lo[14 + cc]);
                        }
                    }
                }
            if (t0 == 0 && !whole) {
                // the item goes on in the CTAs up to the one that holds its last tile
                split_tail = true;
                if (lane == 0) {
                    const uint32_t last = u - v + r.units - 1;
                    const uint32_t big = rest * (share + 1);
                    const uint32_t cl = last < big ? last / (share + 1) : rest + (last - big) / share;
                    p.desc[cta] = Desc{static_cast<int>(cl - c) + 1, rb * C::kRows, r.nq * p.group, head, r.q0, {0, 0, 0}};
                }
            }
        }
        u += n;
        v = 0;
        if (u < u1 && ++item >= r.items && b + 1 < a.tab.B) {
            item = 0;
            do r = request_at<C::kRows>(p, ++b);
            while (r.items == 0 && b + 1 < a.tab.B);
        }
    }
    if (warp == 0 && lane == 0 && !split_tail) p.desc[cta].count = 0;
    if (dead && lane == 0)  // the copies in flight land before the CTA exits
        for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
            mbar_wait_for(&bar[i % C::kStages], (i / C::kStages) & 1, kDrainLimitNs);
}

// Joins the parts of the items that were cut: CTA (c, y) takes rows of the item
// that CTA c of the first kernel began, one warp per row.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) join_kernel(const Params p)
{
    constexpr int ROWS = 8 * NT;
    constexpr int E = D / 32;  // channels per lane
    pdl_wait();
    const int cta = static_cast<int>(blockIdx.x);
    const Desc d = p.desc[cta];
    if (d.count == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = static_cast<int>(blockIdx.y) * kWarps + warp;
    const int row = d.first_row + col;
    if (row >= d.rows) return;
    // part 0 is in the first CTA's second slot, part i in CTA c + i's first
    auto slot = [&](int i) { return (2 * static_cast<size_t>(cta + i) + (i == 0 ? 1 : 0)) * ROWS + col; };
    auto part = [&](int i, float (&x)[E]) {
        const float *src = p.part + slot(i) * D + E * lane;
        if constexpr (E == 4) {
            const float4 y = *reinterpret_cast<const float4 *>(src);
            x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
        } else {
            const float2 y = *reinterpret_cast<const float2 *>(src);
            x[0] = y.x; x[1] = y.y;
        }
    };
    // the first parts are on their way while the maximum is taken
    constexpr int kAhead = 8;
    float ahead[kAhead][E];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i < d.count) part(i, ahead[i]);
    float top = -INFINITY;
    for (int i = lane; i < d.count; i += 32) top = fmaxf(top, p.ml[slot(i)].x);
#pragma unroll
    for (int k = 1; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    float l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    auto join = [&](int i, const float (&x)[E]) {
        const float2 ml = p.ml[slot(i)];
        const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
        l += ml.y * f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += x[e] * f;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i < d.count) join(i, ahead[i]);
#pragma unroll 4
    for (int i = kAhead; i < d.count; ++i) {
        float x[E];
        part(i, x);
        join(i, x);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int i = row / p.group;
    __half *dst = p.a.out + (static_cast<int64_t>(d.q0 + i) * p.a.q_heads + d.head * p.group + row - i * p.group) * D + E * lane;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(dst) = pack2(o[0] * inv, o[1] * inv);
}

template <int D, int NT>
cudaError_t configure_one()
{
    return cudaFuncSetAttribute(attend_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Cfg<D, NT>::kSmem));
}

template <int D, int NT>
cudaError_t launch_one(const Params &prm, int num_sms, cudaStream_t st)
{
    using C = Cfg<D, NT>;
    int grid = num_sms * C::kCtasPerSm;
    if (grid > kMaxCtas) grid = kMaxCtas;
    attend_kernel<D, NT><<<grid, kThreads, C::kSmem, st>>>(prm);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, C::kRows / kWarps, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D, NT>, prm);
}

// 8 query rows per key/value head fill one MMA column tile, more take two
constexpr bool narrow(int64_t rows) { return rows <= 8; }

constexpr size_t round256(size_t v) { return (v + 255) / 256 * 256; }
constexpr int kMaxRows = 16;
constexpr size_t kDescBytes = round256(sizeof(Desc) * kMaxCtas);
constexpr size_t kMlBytes = round256(sizeof(float2) * 2 * kMaxCtas * kMaxRows);

}  // namespace

cudaError_t configure_kv4_attend()
{
    const cudaError_t r[] = {configure_one<128, 1>(), configure_one<128, 2>(), configure_one<64, 1>(), configure_one<64, 2>()};
    for (cudaError_t x : r)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

bool kv4_attend_countable(int64_t B, int64_t heads, int64_t rows, int64_t tokens)
{
    const int64_t item = narrow(rows) ? 8 : kMaxRows;
    return B * heads * ((rows + item - 1) / item) <= UINT32_MAX / ((tokens + kTile - 1) / kTile + kItemCost);
}

size_t kv4_attend_workspace(int D)
{
    return kDescBytes + kMlBytes + sizeof(float) * 2 * kMaxCtas * kMaxRows * static_cast<size_t>(D);
}

cudaError_t launch_kv4_attend(const Kv4AttendArgs &a, int64_t max_rows, void *ws, int num_sms, cudaStream_t st)
{
    uint8_t *w = static_cast<uint8_t *>(ws);
    Params prm{};
    prm.a = a;
    prm.desc = reinterpret_cast<Desc *>(w);
    prm.ml = reinterpret_cast<float2 *>(w + kDescBytes);
    prm.part = reinterpret_cast<float *>(w + kDescBytes + kMlBytes);
    prm.group = a.q_heads / a.cache.heads;
    prm.max_rows = max_rows;
    prm.uk = unpack_consts();
    const int64_t rows = static_cast<int64_t>(a.max_new) * prm.group;
    const bool one = narrow(rows < max_rows ? rows : max_rows);
    if (a.cache.D == 128)
        return one ? launch_one<128, 1>(prm, num_sms, st) : launch_one<128, 2>(prm, num_sms, st);
    return one ? launch_one<64, 1>(prm, num_sms, st) : launch_one<64, 2>(prm, num_sms, st);
}

}  // namespace awq
