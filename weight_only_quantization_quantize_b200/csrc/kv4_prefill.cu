// kv4_prefill.cu -- attention over the paged 4-bit key/value cache for many
// query rows per key/value head (prompts and chunks of prompts): the
// tensor-bound regime, on the 5th-generation tensor cores.
//
//   S = Q C_k^T, p = exp2(step_k scale log2(e) S - m), O = (p step_v) C_v / sum p
// with the integer codes minus zero points C (exact in binary16): the steps
// multiply the logits and the weights in float, one multiply-add and one
// multiply per element, and never enter the tensor cores' operands.
// Roundings: p step_v to binary16 (the second product's operand), the output.
//
// One CTA = 256 query rows (query tokens times the heads of a group, so that a
// tile of codes is unpacked once for all of them) of one key/value head, as two
// 128-row tiles that take turns: while the tensor cores work for one, the
// softmax of the other runs.  Keys come in tiles of 128 tokens.
//   warps 0..3, 4..7   softmax of query tile 0 and 1, one row per thread:
//                      logits from tensor memory, weights back into the same
//                      columns (the second product takes them from there)
//   warps 8..11        unpack: one token per thread, 64 bytes of key and of value
//                      codes straight from global memory (the next tile's are in
//                      registers while this one is written), into two swizzled
//                      shared-memory buffers each
//   warp 12            issues the MMAs (128 x 128 x 16 and 128 x D x 16), the query
//                      tiles in turn: that keeps their softmaxes apart (an issuer per
//                      tile lets them fall into step, 383 -> 394 us for three
//                      prompts of up to 4001 tokens); three more warps fill the warpgroup
// Tensor memory: logits 2 x 128 columns, outputs 2 x D columns.  Values stay in
// token order [token][channel]: the second product reads them as an MN-major
// operand, so nothing is transposed.
//
// The row maximum is not computed: the weights use a standing reference.  The sum
// of a tile's weights, times the largest value step of the tile, tells whether
// one could have left binary16; only then (or while a row has no reference yet, or
// under a mask) a warp looks for the maximum, moves the reference, rescales its
// output rows and computes the weights again.
#include <algorithm>
#include <type_traits>

#include "awq_kernels.cuh"
#include "kv4.cuh"

namespace awq {
namespace {

constexpr int kRowsTile = 128;           // query rows per MMA tile
constexpr int kRowsCta = 2 * kRowsTile;
constexpr int kKeys = 128;               // tokens per tile
constexpr int kStages = 2;
constexpr int kSoftmaxWarps = 8;
constexpr int kUnpackWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps + kUnpackWarps;
constexpr int kThreads = 512;            // the issuer's warpgroup has three idle warps
// registers per thread of each warpgroup; the launch gives 128 to every thread
constexpr int kSoftmaxRegs = 168, kUnpackRegs = 104, kIssueRegs = 72;
static_assert(256 * kSoftmaxRegs + 128 * kUnpackRegs + 128 * kIssueRegs <= kThreads * 128, "register shares");
// log2 of the largest weight, steps included, after an update; of the one that
// asks for the next; and the sum of half a tile's weights below which none can
// be above it (binary16 ends at 65504).  A higher gain trips over the sums: 9
// took three prompts of up to 4001 tokens from 335 to 452 us.
constexpr float kGain = 6.0f, kSlack = 15.0f, kLimit = 46340.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPanel = kKeys * 128;      // bytes of 128 rows x 64 binary16, 128-byte swizzle

template <int D>
struct Cfg {
    static constexpr int kPanels = D / 64;
    static constexpr int kTile = kPanels * kPanel;                 // a Q, K or V tile
    static constexpr int kOCol = 2 * kKeys;                        // output columns after the logits
    static constexpr int kTmemCols = 512;
    static constexpr int kStepBytes = kStages * 2 * kKeys * 4;     // step_k scale log2(e), step_v
    static constexpr size_t kSmem = 1024 + (2 + 2 * kStages) * kTile + kStepBytes + 256;
};

// What the joining kernel has to know of a row block.
struct BlockRows {
    int q0, first, rows, pad;  // the request's first query row; the block's first row; the request's rows
};

struct Params {
    Kv4AttendArgs a;
    int group;
    int splits;      // parts of every row block's keys, one CTA each
    BlockRows *rows; // splits > 1, [row block]
    float2 *ml;      // [row block][head][split][256]: (reference, sum) of a row
    float *part;     // [row block][head][split][256][D]: its numerators
    UnpackConsts uk;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// two floats at a time
__device__ __forceinline__ uint64_t two(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 both(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 32 columns of tensor memory on their way into r; r may be used after
// tmem_arrived(r).
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// codes minus zero point of nibbles 0, 4 (low) or 1, 5 (high) of w
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

// MN-major operand: rows of 64 consecutive n (128 bytes, swizzled), one row per
// k; 8 rows make an atom, atoms 1024 bytes apart along k and kPanel along n.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(kPanel >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Barriers, in shared memory.
struct Bars {
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t q_full[2], s_full[2], p_half[2][2], pv_half[2], o_full[2], drain;
};

// An upper bound of log2(step), at most 1 above it, and that of the smallest step for
// 0 (a slot never written): without the floor a reference of 2^-126 would make
// the weights of such keys infinite.  (Binary16 steps are normal floats, or 0.)
__device__ __forceinline__ float step_log2(float step)
{
    return static_cast<float>(max(static_cast<int>(__float_as_uint(step) >> 23) - 126, -23));
}

template <int N>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const Params p)
{
    using C = Cfg<D>;
    constexpr int W = D / 8;  // packed words of a row
    extern __shared__ uint8_t smem_dyn[];
    const uint32_t raw = smem_u32(smem_dyn);
    uint8_t *smem = smem_dyn + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *sq = smem, *sk = sq + 2 * C::kTile, *sv = sk + kStages * C::kTile;
    float *steps = reinterpret_cast<float *>(sv + kStages * C::kTile);
    __shared__ Bars bars;
    __shared__ uint32_t s_valid[kStages][4];  // tokens of the tile that are there
    __shared__ __align__(16) float s_vmax[kStages][4];  // the largest step of their values, by unpack warp
    __shared__ uint32_t s_tmem;

    const Kv4AttendArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---------------------------------------------------------------- this CTA's rows and keys
    // Row blocks of 256 rows, request after request, and in each the last one
    // first (it sees the most keys).  blockIdx.x counts them for the requests
    // that are this kernel's, found by a scan over all requests.
    const int head = static_cast<int>(blockIdx.y);
    const int flat = static_cast<int>(blockIdx.x) / p.splits, split = static_cast<int>(blockIdx.x) % p.splits;
    __shared__ int s_warp[kThreads / 32], s_request, s_block;
    auto rows_of = [&](int b) -> int {  // of request b, 0 when it is not this kernel's
        const int q0 = a.tab.cu ? a.tab.cu[b] : b;
        const long long q1 = a.tab.cu ? a.tab.cu[b + 1] : b + 1, n = q1 - q0;
        if (q0 < 0 || n < 0 || q1 > a.T || n > a.max_new) {
            if (blockIdx.x == 0 && head == 0) report(a.status, AWQ_ERR_RANGE);
            return 0;
        }
        const long long rows = n * p.group;
        return rows > kPromptRows ? static_cast<int>(rows) : 0;
    };
    {
        if (threadIdx.x == 0) s_request = -1;
        const int per = (a.tab.B + kThreads - 1) / kThreads, b0 = static_cast<int>(threadIdx.x) * per;
        int mine = 0;
        for (int i = 0; i < per && b0 + i < a.tab.B; ++i) mine += (rows_of(b0 + i) + kRowsCta - 1) / kRowsCta;
        int pre = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, pre, d);
            if (lane >= d) pre += y;
        }
        if (lane == 31) s_warp[warp] = pre;
        __syncthreads();
        for (int i = 0; i < warp; ++i) pre += s_warp[i];
        pre -= mine;
        if (flat >= pre && flat < pre + mine) {
            int rem = flat - pre, b = b0, n = (rows_of(b) + kRowsCta - 1) / kRowsCta;
            while (rem >= n && b + 1 < a.tab.B) {
                rem -= n;
                n = (rows_of(++b) + kRowsCta - 1) / kRowsCta;
            }
            s_request = b;
            s_block = n - 1 - rem;
        }
        __syncthreads();
    }
    const int b = s_request;
    if (b < 0) {
        // every field: the join adds to `first` before it compares with `rows`, and the workspace may hold anything
        if (p.splits > 1 && head == 0 && split == 0 && threadIdx.x == 0) p.rows[flat] = BlockRows{0, 0, 0, 0};
        return;
    }
    const int rb = s_block;
    const long long most = static_cast<long long>(a.tab.max_pages) << a.cache.page_shift;
    int len = a.tab.lens[b];
    const int q0 = a.tab.cu ? a.tab.cu[b] : b;
    const int rows = rows_of(b), nq = rows / p.group;
    if (threadIdx.x == 0 && head == 0 && split == 0 && (len < 0 || len > most)) report(a.status, AWQ_ERR_RANGE);
    len = len < 0 ? 0 : len > most ? static_cast<int>(most) : len;
    const int row0 = rb * kRowsCta;
    if (p.splits > 1 && head == 0 && split == 0 && threadIdx.x == 0) p.rows[flat] = BlockRows{q0, row0, rows, 0};
    const int ntiles_q = row0 + kRowsTile < rows ? 2 : 1;
    const int rlast = min(row0 + kRowsCta, rows) - 1;
    const int pfirst = max(len - nq + row0 / p.group, -1);  // positions; -1: before the first token
    const int plast = max(len - nq + rlast / p.group, -1);
    const int lo_first = a.window > 0 ? max(pfirst - a.window + 1, 0) : 0;
    // this split's share of the key tiles
    const int all0 = lo_first / kKeys;
    const int all = plast < 0 ? 0 : plast / kKeys + 1 - all0;
    const int share = (all + p.splits - 1) / p.splits;
    const int tile0 = all0 + min(split * share, all);
    const int tiles = min(share, all - (tile0 - all0));

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.k_full[i], kUnpackWarps);
            mbar_init(&bars.k_empty[i], 1 + 4 * ntiles_q);  // MMA commit, and the softmax warps (steps read)
            mbar_init(&bars.v_full[i], kUnpackWarps);
            mbar_init(&bars.v_empty[i], 1);                 // MMA commit
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars.s_full[t], 1);
            mbar_init(&bars.p_half[t][0], 4);
            mbar_init(&bars.p_half[t][1], 4);
            mbar_init(&bars.pv_half[t], 1);
            mbar_init(&bars.q_full[t], 4);
            mbar_init(&bars.o_full[t], 1);
        }
        mbar_init(&bars.drain, 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(C::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp < kSoftmaxWarps) {
        // ------------------------------------------------------------ softmax
        more_registers<kSoftmaxRegs>();
        const int t = warp >> 2;
        if (t < ntiles_q) {
            const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
            const uint32_t ts = tmem + lanes + t * kKeys;
            const uint32_t to = tmem + lanes + C::kOCol + t * D;
            const int r = 32 * (warp & 3) + lane;  // row of the tile
            const int row = row0 + t * kRowsTile + r;
            const bool in = row < rows;
            const int qi = in ? row / p.group : 0;
            const int qh = head * p.group + (in ? row - qi * p.group : 0);
            // The warp's 32 query rows into the swizzled tile, W lanes per row,
            // channels of each 8 in the order (0,4),(1,5),(2,6),(3,7) that the
            // unpack gives the keys.
            {
                const int c = lane % W;
                uint4 x[W];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const int rr = 32 * (warp & 3) + i * (32 / W) + lane / W;
                    const int rw = row0 + t * kRowsTile + rr;
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (rw < rows) {
                        const int ri = rw / p.group;
                        const int rh = head * p.group + rw - ri * p.group;
                        x[i] = __ldg(reinterpret_cast<const uint4 *>(a.q + (q0 + ri) * a.q_stride + static_cast<int64_t>(rh) * D) + c);
                    }
                }
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const int rr = 32 * (warp & 3) + i * (32 / W) + lane / W;
                    uint8_t *dst = sq + t * C::kTile + rr * 128 + (c >> 3) * kPanel + (((c & 7) ^ (rr & 7)) << 4);
                    *reinterpret_cast<uint4 *>(dst) =
                        make_uint4(__byte_perm(x[i].x, x[i].z, 0x5410), __byte_perm(x[i].x, x[i].z, 0x7632),
                                   __byte_perm(x[i].y, x[i].w, 0x5410), __byte_perm(x[i].y, x[i].w, 0x7632));
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.q_full[t]);
            }
            const int pos = in ? max(len - nq + qi, -1) : -1;
            const int lo = a.window > 0 ? pos - a.window : -1;
            // positions of the tile's first and last row: a key tile that every
            // row sees needs no mask
            const int rt = row0 + t * kRowsTile, re = min(rt + kRowsTile, rows) - 1;
            const int p_lo = max(len - nq + rt / p.group, -1);
            const int w_hi = a.window > 0 ? max(len - nq + re / p.group, -1) - a.window : -1;
            float m = in ? -INFINITY : 0.0f, l = 0.0f;
            bool ok = true, ready = false;
            for (int j = 0; j < tiles; ++j) {
                const int st = j % kStages;
                const uint32_t ph = (j / kStages) & 1;
                bool w = mbar_wait(&bars.k_full[st], ph);  // the steps
                if (w) w = mbar_wait(&bars.s_full[t], j & 1);
                if (!__all_sync(0xffffffffu, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float *ks = steps + st * 2 * kKeys, *vs = ks + kKeys;
                const int tok = (tile0 + j) * kKeys;
                const bool clear = (s_valid[st][0] & s_valid[st][1] & s_valid[st][2] & s_valid[st][3]) == 0xffffffffu && tok + kKeys - 1 <= p_lo && tok > w_hi;
                const float4 vm4 = *reinterpret_cast<const float4 *>(s_vmax[st]);
                const float vmax = fmaxf(fmaxf(vm4.x, vm4.y), fmaxf(vm4.z, vm4.w));
                // the weights of half h, as far as they are stored, go to the second product
                auto publish = [&](int h) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.p_half[t][h]);
                };
                // which of the n (16 or 32) keys from tok + c0 on are there and seen: lo < key <= pos
                auto seen_of = [&](int c0, int n) -> uint32_t {
                    const int up = pos - tok - c0, dn = lo - tok - c0;
                    uint32_t seen = up < 0 ? 0u : up >= 31 ? 0xffffffffu : (2u << up) - 1u;
                    if (dn >= 0) seen &= dn >= 31 ? 0u : ~((2u << dn) - 1u);
                    return seen & (s_valid[st][c0 / 32] >> (n == 16 ? c0 & 16 : 0));
                };
                // Keys h0 .. h0 + 63 with masks: the maximum, the reference, the output
                // rows, the weights, 16 keys at a time.
                auto masked_half = [&](int h0) -> bool {
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c0 = h0; c0 < h0 + 64; c0 += 16) {
                        uint32_t y[16];
                        tmem_ld16(ts + c0, y);
                        const uint32_t seen = seen_of(c0, 16);
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if ((seen >> c) & 1u) top = fmaxf(top, fmaf(__uint_as_float(y[c]), ks[c0 + c], step_log2(vs[c0 + c])));
                    }
                    float f = 1.0f;
                    if (top > m + kSlack) {
                        const float next = top - kGain;
                        f = ex2(m - next);  // 0 for the first one
                        m = next;
                        l *= f;
                    }
                    if ((j > 0 || h0 > 0) && __any_sync(0xffffffffu, f != 1.0f)) {
                        // the sums so far: those of earlier tiles were complete before this
                        // tile's logits, the first half's are waited for
                        if (h0 > 0) {
                            if (!__all_sync(0xffffffffu, mbar_wait(&bars.pv_half[t], j & 1))) return false;
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + c0, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(to + c0, o);
                        }
                    }
#pragma unroll 1
                    for (int c0 = h0; c0 < h0 + 64; c0 += 32) {
                        uint32_t z[16];
#pragma unroll
                        for (int g = 0; g < 32; g += 16) {
                            uint32_t y[16];
                            tmem_ld16(ts + c0 + g, y);
                            const uint32_t seen = seen_of(c0 + g, 16);
#pragma unroll
                            for (int c = 0; c < 16; c += 2) {
                                float pv[2];
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    // select, never multiply: a masked place gives 0
                                    const bool in_sight = (seen >> (c + h)) & 1u;
                                    const float e = in_sight ? ex2(fmaf(__uint_as_float(y[c + h]), ks[c0 + g + c + h], -m)) : 0.0f;
                                    l += e;
                                    pv[h] = in_sight ? e * vs[c0 + g + c + h] : 0.0f;
                                }
                                z[(g + c) / 2] = pack2(pv[0], pv[1]);
                            }
                        }
                        tmem_st16(ts + c0 / 2, z);  // over logits that have been read
                    }
                    return true;
                };
                if (!ready && clear) {
                    // a first reference from the first 16 keys, good enough unless a weight passes the limit
                    uint32_t y[16];
                    tmem_ld16(ts, y);
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 16; ++c) top = fmaxf(top, fmaf(__uint_as_float(y[c]), ks[c], step_log2(vs[c])));
                    if (m == -INFINITY) m = top - kGain;
                    ready = __all_sync(0xffffffffu, m > -INFINITY);
                }
                // Half the tile at a time: the second product starts on the first 64
                // weights while the others are computed.
                uint32_t x[2][32];
                if (ready) tmem_ld32_start(ts, x[0]);
                // Weights of half h with the reference as it stands; true when one may be too large (then nothing is stored).
                auto weights = [&](auto mask, int h) -> bool {
                    constexpr bool MASK = decltype(mask)::value;
                    const int h0 = 64 * h;
                    uint32_t pk[32];
                    uint64_t sum0 = 0, sum1 = 0;
                    const uint64_t nm = two(-m, -m);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        // the next 32 logits are on their way while these are worked on
                        tmem_arrived(x[g]);
                        const uint32_t seen = MASK ? seen_of(h0 + 32 * g, 32) : 0u;
                        if (h0 + 32 * g + 32 < kKeys) tmem_ld32_start(ts + h0 + 32 * g + 32, x[1 - g]);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const int k = h0 + 32 * g + c;
                            const ulonglong2 kf = *reinterpret_cast<const ulonglong2 *>(ks + k);
                            const ulonglong2 vf = *reinterpret_cast<const ulonglong2 *>(vs + k);
                            float2 y0 = both(fma2(two(__uint_as_float(x[g][c]), __uint_as_float(x[g][c + 1])), kf.x, nm));
                            float2 y1 = both(fma2(two(__uint_as_float(x[g][c + 2]), __uint_as_float(x[g][c + 3])), kf.y, nm));
                            if constexpr (MASK) {  // weight 0 (absent keys have codes and steps 0: nothing here is NaN)
                                y0.x = (seen >> c) & 1u ? y0.x : -INFINITY;
                                y0.y = (seen >> (c + 1)) & 1u ? y0.y : -INFINITY;
                                y1.x = (seen >> (c + 2)) & 1u ? y1.x : -INFINITY;
                                y1.y = (seen >> (c + 3)) & 1u ? y1.y : -INFINITY;
                            }
                            const uint64_t e0 = two(ex2(y0.x), ex2(y0.y)), e1 = two(ex2(y1.x), ex2(y1.y));
                            sum0 = add2(sum0, e0);
                            sum1 = add2(sum1, e1);
                            const float2 w0 = both(mul2(e0, vf.x)), w1 = both(mul2(e1, vf.y));
                            pk[16 * g + c / 2] = pack2(w0.x, w0.y);
                            pk[16 * g + c / 2 + 1] = pack2(w1.x, w1.y);
                        }
                        if (h == 1 && g == 0) publish(0);  // the first half's weights have arrived by now
                    }
                    const float2 s2 = both(add2(sum0, sum1));
                    const float sum = s2.x + s2.y;
                    const bool over = __any_sync(0xffffffffu, !(sum * vmax <= kLimit));
                    if (!over) {
                        l += sum;
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t z[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) z[i] = pk[16 * g + i];
                            tmem_st16(ts + 32 * h + 16 * g, z);
                        }
                    }
                    return over;
                };
                // The usual tile first, in one piece of code; what is left of it (masks, a
                // weight over the limit, no reference yet) in another, once for both halves.
                int from = 0;
                if (ready && clear && !weights(std::false_type{}, 0)) from = weights(std::false_type{}, 1) ? 1 : 2;
#pragma unroll 1
                for (int h = from; h < 2; ++h) {
                    if (!ready && h == 1) publish(0);
                    // the half that has just failed goes on to its maximum
                    if (!ready || (clear && h == from) || weights(std::true_type{}, h)) ok = masked_half(64 * h) && ok;
                }
                // after a wait that ran out too: the issuer then goes on with whatever the
                // columns hold, and drains it (a branch around this: 338 -> 341 us)
                publish(1);
                if (lane == 0) mbar_arrive(&bars.k_empty[st]);
                if (!ok) break;
                if (!ready) ready = __all_sync(0xffffffffu, m != -INFINITY);
            }
            // -------------------------------------------------------- output
            if (tiles > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_full[t], 0));
            if (!ok) {
                if (lane == 0) report(a.status, AWQ_ERR_DEVICE_TIMEOUT);
            } else {
                tc_fence_after();
                if (p.splits > 1) {
                    // numerators, reference and sum for the join
                    const size_t at = (static_cast<size_t>(flat) * gridDim.y + head) * p.splits + split;
                    const size_t slot = at * kRowsCta + t * kRowsTile + r;
                    if (in) p.ml[slot] = make_float2(m, l);
#pragma unroll 1
                    for (int c0 = 0; c0 < D && tiles > 0; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32_start(to + c0, o);
                        tmem_arrived(o);
                        if (!in) continue;
#pragma unroll
                        for (int c = 0; c < 32; c += 8) {
                            // columns hold channels 0, 4, 1, 5, 2, 6, 3, 7 of each 8
                            uint4 *dst = reinterpret_cast<uint4 *>(p.part + slot * D + c0 + c);
                            dst[0] = make_uint4(o[c], o[c + 2], o[c + 4], o[c + 6]);
                            dst[1] = make_uint4(o[c + 1], o[c + 3], o[c + 5], o[c + 7]);
                        }
                    }
                }
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                uint4 *dst = reinterpret_cast<uint4 *>(a.out + (static_cast<int64_t>(q0 + qi) * a.q_heads + qh) * D);
#pragma unroll 1
                for (int c0 = 0; c0 < D && p.splits == 1; c0 += 32) {
                    uint32_t o[32];
                    if (tiles > 0)
                        tmem_ld32(to + c0, o);
                    else
#pragma unroll
                        for (int c = 0; c < 32; ++c) o[c] = 0u;
                    if (in) {
#pragma unroll
                        for (int c = 0; c < 32; c += 8) {
                            // columns hold channels 0, 4, 1, 5, 2, 6, 3, 7 of each 8
                            float x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(o[c + i]) * inv;
                            dst[(c0 + c) / 8] = make_uint4(pack2(x[0], x[2]), pack2(x[4], x[6]), pack2(x[1], x[3]), pack2(x[5], x[7]));
                        }
                    }
                }
            }
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ unpack
        fewer_registers<kUnpackRegs>();
        const int uw = warp - kSoftmaxWarps;
        const int tok_in = 32 * uw + lane;  // token of the tile
        const int sh = a.cache.page_shift - 4;
        const int32_t *table = a.tab.block_table + static_cast<size_t>(b) * a.tab.max_pages;
        const float c1 = a.scale * kLog2e;
        const UnpackConsts uk = p.uk;
        const int end = min(len, plast + 1);  // keys from here on are seen by no row
        // codes and steps of tile j's token; false where there is none
        auto fetch = [&](int j, uint4 (&kx)[W / 4], uint4 (&vx)[W / 4], uint32_t &km, uint32_t &vm) -> bool {
            const int tok = (tile0 + j) * kKeys + tok_in;
            bool there = j < tiles && tok < end && tok >= lo_first;  // pages before the window may be gone
            if (there) {
                const int page = table[tok >> a.cache.page_shift];
                if (page < 0 || page >= a.cache.num_pages) {
                    report(a.status, AWQ_ERR_RANGE);
                    there = false;
                } else {
                    const int64_t block = ((static_cast<int64_t>(page) * a.cache.heads + head) << sh) + ((tok >> 4) & ((1 << sh) - 1));
                    const uint8_t *src = a.cache.data + block * kv4_block_bytes(D);
                    const uint4 *kr = reinterpret_cast<const uint4 *>(src + (tok & 15) * (D / 2));
                    const uint4 *vr = reinterpret_cast<const uint4 *>(src + 8 * D + (tok & 15) * (D / 2));
#pragma unroll
                    for (int i = 0; i < W / 4; ++i) {
                        kx[i] = kr[i];
                        vx[i] = vr[i];
                    }
                    km = *reinterpret_cast<const uint32_t *>(src + 16 * D + 4 * (tok & 15));
                    vm = *reinterpret_cast<const uint32_t *>(src + 16 * D + 64 + 4 * (tok & 15));
                }
            }
            if (!there) {
                // zero codes at zero point 0: finite, and masked by s_valid
#pragma unroll
                for (int i = 0; i < W / 4; ++i) kx[i] = vx[i] = make_uint4(0, 0, 0, 0);
                km = vm = 0;
            }
            return there;
        };
        auto unpack = [&](uint8_t *tile, const uint4 (&x)[W / 4], uint32_t meta) {
            const uint32_t z = (meta >> 16) & 15u;
            uint32_t za, zb;
            zero_constants(z, za, zb);
            uint8_t *dst = tile + tok_in * 128;
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = 4 * i + k;
                    const uint32_t w8 = w[k] >> 8;
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * kPanel + (((c & 7) ^ (tok_in & 7)) << 4)) =
                        make_uint4(codes_low(w[k], za, uk), codes_high(w[k], zb, uk), codes_low(w8, za, uk), codes_high(w8, zb, uk));
                }
            }
        };
        bool ok = true;
        uint4 kx[W / 4], vx[W / 4];
        uint32_t km = 0, vm = 0;
        bool there = fetch(0, kx, vx, km, vm);
        for (int j = 0; j < tiles; ++j) {
            const int st = j % kStages;
            const uint32_t ph = ((j / kStages) & 1) ^ 1u;
            uint4 kn[W / 4], vn[W / 4];
            uint32_t kmn, vmn;
            const bool next = fetch(j + 1, kn, vn, kmn, vmn);
            bool w = j < kStages || mbar_wait(&bars.k_empty[st], ph);
            if (!__all_sync(0xffffffffu, w)) {
                ok = false;
                break;
            }
            float *ks = steps + st * 2 * kKeys;
            ks[tok_in] = __half2float(__ushort_as_half(static_cast<uint16_t>(km))) * c1;
            ks[kKeys + tok_in] = __half2float(__ushort_as_half(static_cast<uint16_t>(vm)));
            const uint32_t valid = __ballot_sync(0xffffffffu, there);
            const uint32_t vtop = __reduce_max_sync(0xffffffffu, vm & 0xffffu);  // steps are positive: ordered as integers
            if (lane == 0) {
                s_valid[st][uw] = valid;
                s_vmax[st][uw] = __half2float(__ushort_as_half(static_cast<uint16_t>(vtop)));
            }
            unpack(sk + st * C::kTile, kx, km);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.k_full[st]);
            w = j < kStages || mbar_wait(&bars.v_empty[st], ph);
            if (!__all_sync(0xffffffffu, w)) {
                ok = false;
                break;
            }
            unpack(sv + st * C::kTile, vx, vm);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.v_full[st]);
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                kx[i] = kn[i];
                vx[i] = vn[i];
            }
            km = kmn;
            vm = vmn;
            there = next;
        }
        if (!ok && lane == 0) report(a.status, AWQ_ERR_DEVICE_TIMEOUT);
    } else {
        // ------------------------------------------------------------ MMA issuer
        fewer_registers<kIssueRegs>();
        if (warp == kMmaWarp && lane == 0 && tiles > 0) {
            constexpr uint32_t id_s = tc_idesc_f16(kRowsTile, kKeys);
            constexpr uint32_t id_o = tc_idesc_f16(kRowsTile, D) | (1u << 16);  // B is MN-major
            // Descriptors are made once and moved by adding to their address field: the
            // issuing thread shares its scheduler with three busy warps, and every
            // instruction between two MMAs shows.
            const uint64_t q_desc = sw128_desc(smem_u32(sq)), k_desc = sw128_desc(smem_u32(sk)), v_desc = mn_desc(smem_u32(sv));
            auto logits = [&](int t, int st) {
                const uint64_t qd = q_desc + t * (C::kTile >> 4), kd = k_desc + st * (C::kTile >> 4);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = ((s >> 2) * kPanel + 32 * (s & 3)) >> 4;
                    tc_mma(tmem + t * kKeys, qd + off, kd + off, id_s, s > 0 ? 1u : 0u);
                }
                tc_commit(&bars.s_full[t]);
            };
            bool ok = mbar_wait(&bars.k_full[0], 0);
            for (int t = 0; t < ntiles_q && ok; ++t) {
                ok = mbar_wait(&bars.q_full[t], 0);
                if (!ok) break;
                tc_fence_after();
                logits(t, 0);
            }
            if (ok) tc_commit(&bars.k_empty[0]);
            for (int j = 0; j < tiles && ok; ++j) {
                const int st = j % kStages, sn = (j + 1) % kStages;
                ok = mbar_wait(&bars.v_full[st], (j / kStages) & 1);
                for (int t = 0; t < ntiles_q && ok; ++t) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && mbar_wait(&bars.p_half[t][h], j & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t w = tmem + t * kKeys + 32 * h, to = tmem + C::kOCol + t * D;
                        const uint64_t vd = v_desc + st * (C::kTile >> 4) + h * (8192 >> 4);
                        tc_mma_ta(to, w, vd, id_o, j > 0 || h > 0 ? 1u : 0u);
#pragma unroll
                        for (int s = 1; s < kKeys / 32; ++s) tc_mma_ta(to, w + 8 * s, vd + s * (2048 >> 4), id_o, 1u);
                        if (h == 0) tc_commit(&bars.pv_half[t]);
                    }
                    if (!ok) break;
                    if (t == ntiles_q - 1) tc_commit(&bars.v_empty[st]);
                    if (j + 1 == tiles) {
                        tc_commit(&bars.o_full[t]);
                        continue;
                    }
                    if (t == 0) ok = mbar_wait(&bars.k_full[sn], ((j + 1) / kStages) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    logits(t, sn);
                }
                if (ok && j + 1 < tiles) tc_commit(&bars.k_empty[sn]);
            }
            if (!ok) report(a.status, AWQ_ERR_DEVICE_TIMEOUT);
            // Every MMA issued completes, and every commit has arrived, before tensor
            // memory is freed and the CTA leaves, whichever role's wait ran out (the
            // softmax warps skip the outputs' barrier after one of theirs).  Otherwise it
            // passes with that barrier.
            tc_commit(&bars.drain);
            mbar_wait_for(&bars.drain, 0, kDrainLimitNs);
        }
    }
    __syncwarp();

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
    }
}

// Joins the splits of a row block, one warp per row, in the order of the splits.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const Params p)
{
    constexpr int E = D / 32;
    pdl_wait();
    const Kv4AttendArgs &a = p.a;
    const int flat = static_cast<int>(blockIdx.x) / (kRowsCta / 8), head = static_cast<int>(blockIdx.y);
    const int r = static_cast<int>(blockIdx.x) % (kRowsCta / 8) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const BlockRows br = p.rows[flat];
    const int row = br.first + r;
    if (row >= br.rows) return;
    const size_t first = (static_cast<size_t>(flat) * gridDim.y + head) * p.splits;
    auto slot = [&](int s) { return (first + s) * kRowsCta + r; };
    float top = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) top = fmaxf(top, p.ml[slot(s)].x);
#pragma unroll
    for (int k = 1; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    float l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        const float2 ml = p.ml[slot(s)];
        // A part that saw no key has the sum 0, and its numerators may not be written.  (A
        // row of NaN logits has no reference either, but a sum of NaN, which has to reach
        // the output.)
        if (ml.y == 0.0f) continue;
        const float f = ex2(ml.x - top);  // NaN for a row without a reference: like its sum
        l += ml.y * f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += p.part[slot(s) * D + E * lane + e] * f;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int qi = row / p.group;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + (static_cast<int64_t>(br.q0 + qi) * a.q_heads + head * p.group +
                                                           row - qi * p.group) * D + E * lane);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack2(o[e] * inv, o[e + 1] * inv);
}

// Partial results that the workspace holds, 256 rows each.
constexpr int kMaxParts = 160;
constexpr size_t kBlockBytes = (sizeof(BlockRows) * kMaxParts + 255) / 256 * 256;
constexpr size_t kMlBytes = sizeof(float2) * kMaxParts * kRowsCta;

}  // namespace

size_t kv4_prefill_workspace(int D)
{
    return kBlockBytes + kMlBytes + sizeof(float) * kMaxParts * kRowsCta * static_cast<size_t>(D);
}

cudaError_t configure_kv4_prefill()
{
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(Cfg<128>::kSmem));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(prefill_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Cfg<64>::kSmem));
}

cudaError_t launch_kv4_prefill(const Kv4AttendArgs &a, void *ws, int num_sms, cudaStream_t st)
{
    Params prm{};
    prm.a = a;
    prm.group = a.q_heads / a.cache.heads;
    prm.uk = unpack_consts();
    // Row blocks at most: T queries in whole blocks, and one cut block for each
    // request that has enough rows to be this kernel's.
    const int64_t all = a.T * prm.group, of_one = (std::min<int64_t>(a.max_new, a.T) * prm.group + kRowsCta - 1) / kRowsCta;
    const int64_t requests = std::min<int64_t>(a.tab.B, all / (kPromptRows + 1));
    const int64_t bound = std::min(all / kRowsCta + requests, of_one * a.tab.B);
    if (bound == 0) return cudaSuccess;  // too few queries for any such request
    // Few row blocks leave SMs idle: their keys are split until the GPU is full,
    // into parts of at least four tiles (by the table's width, the only length
    // known here).
    const int64_t blocks = bound * a.cache.heads;
    const int sms = num_sms < kMaxParts ? num_sms : kMaxParts;
    const int64_t by_keys = (static_cast<int64_t>(a.tab.max_pages) << a.cache.page_shift) / (4 * kKeys);
    int64_t splits = blocks < sms ? sms / blocks : 1;
    if (splits > by_keys) splits = by_keys < 1 ? 1 : by_keys;
    prm.splits = static_cast<int>(splits);
    uint8_t *w = static_cast<uint8_t *>(ws);
    prm.rows = reinterpret_cast<BlockRows *>(w);
    prm.ml = reinterpret_cast<float2 *>(w + kBlockBytes);
    prm.part = reinterpret_cast<float *>(w + kBlockBytes + kMlBytes);
    const dim3 grid(static_cast<unsigned>(bound * splits), static_cast<unsigned>(a.cache.heads));
    if (a.cache.D == 128)
        prefill_kernel<128><<<grid, kThreads, Cfg<128>::kSmem, st>>>(prm);
    else
        prefill_kernel<64><<<grid, kThreads, Cfg<64>::kSmem, st>>>(prm);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || prm.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(bound) * (kRowsCta / 8), grid.y, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.cache.D == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<128>, prm) : cudaLaunchKernelEx(&cfg, join_kernel<64>, prm);
}

}  // namespace awq
