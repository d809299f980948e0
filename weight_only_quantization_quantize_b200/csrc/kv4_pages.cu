// kv4_pages.cu -- block tables and slot maps of the paged 4-bit cache, built
// on the GPU from request lengths.
//
// reserve: request b holds ceil(len_b / P) pages and gets new_b tokens, so it
// needs need_b = ceil((len_b + new_b) / P) - ceil(len_b / P) more.  With
// first_b = sum of need over the earlier requests, its k-th new page is
//   free_pages[free_count - 1 - (first_b + k)]
// (the free pages are a stack), and token i of request b goes to
//   slot = table[b, (len_b + i) / P] P + (len_b + i) mod P.
//
// Launch-bound: a decode step reads and writes a few KB.  One launch of one
// thread-block cluster: every CTA scans all requests itself (B <= 4096 words
// from L2) and writes its share of tokens and pages, so nothing passes between
// CTAs but one cluster barrier, after which the lengths and the free count,
// which may be updated in place, are written.  All CTAs decide alike whether
// the call fits, from the same inputs, so a refused call changes nothing.
#include "kv4.cuh"

namespace awq {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxB = AWQ_KV4_MAX_REQUESTS;
constexpr int kPer = kMaxB / kThreads;  // requests per thread at most
constexpr size_t kSmemBytes = sizeof(int32_t) * (3 * static_cast<size_t>(kMaxB) + 2);

struct Pair {
    long long a, b;
};

// Exclusive block scan of one pair per thread; *total receives the sums.
__device__ Pair block_scan(Pair v, Pair *total)
{
    __shared__ Pair warp_sum[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair x = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long ya = __shfl_up_sync(0xffffffffu, x.a, d), yb = __shfl_up_sync(0xffffffffu, x.b, d);
        if (lane >= d) {
            x.a += ya;
            x.b += yb;
        }
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    Pair before{0, 0}, all{0, 0};
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) {
            before.a += warp_sum[w].a;
            before.b += warp_sum[w].b;
        }
        all.a += warp_sum[w].a;
        all.b += warp_sum[w].b;
    }
    __syncthreads();
    *total = all;
    return Pair{before.a + x.a - v.a, before.b + x.b - v.b};
}

// The request b with start[b] <= i < start[b + 1] (start[0] = 0, i < start[n]).
__device__ __forceinline__ int owner_of(const int32_t *start, int n, int i)
{
    int lo = 0, hi = n;  // start[lo] <= i < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct ReserveParams {
    const int32_t *new_lens, *lens, *free_pages, *free_count;
    int32_t *block_table;
    int64_t *slots;
    int32_t *positions, *cu, *lens_out, *free_count_out, *status;
    int64_t num_pages, T;
    int B, page_shift, max_pages;
};

__global__ void __launch_bounds__(kThreads) reserve_kernel(const ReserveParams p)
{
    extern __shared__ int32_t sm[];
    int32_t *s_cu = sm;                // [B + 1] tokens before each request
    int32_t *s_first = sm + p.B + 1;   // [B + 1] new pages before each request
    int32_t *s_len = sm + 2 * p.B + 2; // [B]
    const int rank = static_cast<int>(blockIdx.x), ranks = static_cast<int>(gridDim.x);
    const int P1 = (1 << p.page_shift) - 1;
    const long long most = static_cast<long long>(p.max_pages) << p.page_shift;
    const int free0 = *p.free_count;

    int bad = free0 < 0 || free0 > p.num_pages;
    int len[kPer], nw[kPer];
    Pair mine{0, 0};
    const int per = (p.B + kThreads - 1) / kThreads;  // consecutive requests per thread
    const int b0 = static_cast<int>(threadIdx.x) * per;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        len[j] = nw[j] = 0;
        if (j < per && b0 + j < p.B) {
            len[j] = p.lens[b0 + j];
            nw[j] = p.new_lens[b0 + j];
            if (len[j] < 0 || nw[j] < 0 || static_cast<long long>(len[j]) + nw[j] > most) {
                bad = 1;
                nw[j] = 0;
            }
            mine.a += nw[j];
            if (nw[j] > 0)
                mine.b += ((len[j] + nw[j] - 1) >> p.page_shift) - ((len[j] - 1) >> p.page_shift);
        }
    }
    Pair total;
    Pair at = block_scan(mine, &total);
    bad = __syncthreads_or(bad || total.a > p.T);
    const bool full = total.b > free0;
    const bool ok = !bad && !full;
    if (!ok && rank == 0 && threadIdx.x == 0) report(p.status, bad ? AWQ_ERR_RANGE : AWQ_ERR_CAPACITY);
    if (ok) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < per && b0 + j < p.B) {
                s_cu[b0 + j] = static_cast<int32_t>(at.a);
                s_first[b0 + j] = static_cast<int32_t>(at.b);
                s_len[b0 + j] = len[j];
                at.a += nw[j];
                if (nw[j] > 0)
                    at.b += ((len[j] + nw[j] - 1) >> p.page_shift) - ((len[j] - 1) >> p.page_shift);
            }
        if (threadIdx.x == 0) {
            s_cu[p.B] = static_cast<int32_t>(total.a);
            s_first[p.B] = static_cast<int32_t>(total.b);
        }
    }
    __syncthreads();

    const int64_t stride = static_cast<int64_t>(ranks) * kThreads;
    const int64_t tid = static_cast<int64_t>(rank) * kThreads + threadIdx.x;
    const int tokens = ok ? static_cast<int>(total.a) : 0;
    constexpr int kAhead = 4;  // tokens per turn, whose page lookups are in flight together
    for (int64_t t0 = tid; t0 < p.T; t0 += kAhead * stride) {
        const int32_t *entry[kAhead];
        int pos[kAhead], page[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t t = t0 + i * stride;
            entry[i] = nullptr;
            pos[i] = -1;
            if (t < tokens) {
                const int b = owner_of(s_cu, p.B, static_cast<int>(t));
                pos[i] = s_len[b] + static_cast<int>(t) - s_cu[b];
                const int col = pos[i] >> p.page_shift;
                const int held = (s_len[b] + P1) >> p.page_shift;
                entry[i] = col < held ? p.block_table + static_cast<size_t>(b) * p.max_pages + col
                                      : p.free_pages + (free0 - 1 - (s_first[b] + col - held));
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) page[i] = entry[i] ? *entry[i] : -1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (entry[i] && (page[i] < 0 || page[i] >= p.num_pages)) {  // its tokens have no slot
                page[i] = -1;
                report(p.status, AWQ_ERR_RANGE);
            }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t t = t0 + i * stride;
            if (t >= p.T) break;
            p.slots[t] = page[i] < 0 ? -1 : (static_cast<int64_t>(page[i]) << p.page_shift) + (pos[i] & P1);
            if (p.positions) p.positions[t] = pos[i];
        }
    }
    // the new pages' table entries: read by no thread of this launch
    const int pages = ok ? static_cast<int>(total.b) : 0;
    for (int64_t i = tid; i < pages; i += stride) {
        const int b = owner_of(s_first, p.B, static_cast<int>(i));
        const int held = (s_len[b] + P1) >> p.page_shift;
        const int page = p.free_pages[free0 - 1 - i];  // a bad one has been reported with its tokens
        p.block_table[static_cast<size_t>(b) * p.max_pages + held + (i - s_first[b])] =
            page < 0 || page >= p.num_pages ? -1 : page;
    }
    // every CTA has read the lengths and the free count: they may be replaced
    cluster_arrive_release();
    cluster_wait_acquire();
    for (int64_t b = tid; b <= p.B; b += stride) {
        p.cu[b] = ok ? s_cu[b] : 0;
        if (b < p.B) {
            if (ok)
                p.lens_out[b] = s_len[b] + s_cu[b + 1] - s_cu[b];
            else if (p.lens_out != p.lens)
                p.lens_out[b] = p.lens[b];
        }
    }
    if (tid == 0) *p.free_count_out = ok ? free0 - pages : free0;
}

struct ReleaseParams {
    const int32_t *done;
    int32_t *lens, *block_table, *free_pages, *free_count, *status;
    int64_t num_pages;
    int B, page_shift, max_pages;
};

// One CTA: pushes the pages of the flagged requests, in the order of requests
// and of their table rows, clears those rows and lengths.  Entries of -1 (pages
// that left the window and were given back) are passed over; where there are any,
// every thread counts the pages of a run of entries, and a scan gives their
// places.  Without any, an entry's place is its number: neighbouring threads then
// take neighbouring entries (256 rows of 64 pages 24 us, 32 by runs).
__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseParams p)
{
    extern __shared__ int32_t sm[];
    int32_t *s_first = sm;  // [B + 1]
    const int P1 = (1 << p.page_shift) - 1;
    const int free0 = *p.free_count;
    int bad = free0 < 0 || free0 > p.num_pages;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = static_cast<int>(threadIdx.x) * per;
    int held[kPer];
    Pair mine{0, 0};
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        held[j] = 0;
        if (j < per && b0 + j < p.B && p.done[b0 + j]) {
            const int len = p.lens[b0 + j];
            const long long n = len < 0 ? -1 : (static_cast<long long>(len) + P1) >> p.page_shift;
            if (n < 0 || n > p.max_pages)
                bad = 1;
            else
                held[j] = static_cast<int>(n);
            mine.a += held[j];
        }
    }
    Pair total;
    Pair at = block_scan(mine, &total);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (j < per && b0 + j < p.B) {
            s_first[b0 + j] = static_cast<int32_t>(at.a);
            at.a += held[j];
        }
    if (threadIdx.x == 0) s_first[p.B] = static_cast<int32_t>(total.a);
    bad = __syncthreads_or(bad || total.a > INT32_MAX);
    const int entries = bad ? 0 : static_cast<int>(total.a);
    int lost = 0, gone = 0;  // a page outside the cache; an entry without a page
    for (int i = threadIdx.x; i < entries; i += kThreads) {
        const int b = owner_of(s_first, p.B, i);
        const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + i - s_first[b]];
        lost |= page < -1 || page >= p.num_pages;
        gone |= page < 0;
    }
    gone = __syncthreads_or(gone);
    long long pages = entries;
    const int share = (entries + kThreads - 1) / kThreads;
    const int i0 = static_cast<int>(min(static_cast<long long>(threadIdx.x) * share, pages));
    const int i1 = min(i0 + share, entries);
    auto each = [&](auto f) {  // f(entry) over this thread's run
        int b = i0 < i1 ? owner_of(s_first, p.B, i0) : 0;
        for (int i = i0; i < i1; ++i) {
            while (i >= s_first[b + 1]) ++b;
            f(p.block_table + static_cast<size_t>(b) * p.max_pages + i - s_first[b]);
        }
    };
    Pair before{0, 0};
    if (gone) {
        Pair own{0, 0}, all;
        each([&](const int32_t *e) { own.a += *e >= 0; });
        before = block_scan(own, &all);
        pages = all.a;
    }
    if (__syncthreads_or(lost || bad || pages + free0 > p.num_pages)) {
        if (threadIdx.x == 0) report(p.status, AWQ_ERR_RANGE);
        return;
    }
    if (gone) {
        int32_t *dst = p.free_pages + free0 + before.a;
        each([&](int32_t *e) {
            const int page = *e;
            if (page < 0) return;
            *dst++ = page;
            *e = -1;
        });
    } else {
        for (int i = threadIdx.x; i < entries; i += kThreads) {
            const int b = owner_of(s_first, p.B, i);
            int32_t *e = p.block_table + static_cast<size_t>(b) * p.max_pages + i - s_first[b];
            p.free_pages[free0 + i] = *e;
            *e = -1;
        }
    }
    for (int b = threadIdx.x; b < p.B; b += kThreads)
        if (p.done[b]) p.lens[b] = 0;
    if (threadIdx.x == 0) *p.free_count = free0 + static_cast<int>(pages);
}

}  // namespace

cudaError_t configure_kv4_pages()
{
    cudaError_t e = cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSmemBytes));
}

cudaError_t launch_kv4_reserve(const int32_t *new_lens, const int32_t *lens, int B, int page_shift,
                               int32_t *block_table, int max_pages, const int32_t *free_pages,
                               const int32_t *free_count, int64_t num_pages, int64_t T, int64_t *slots,
                               int32_t *positions, int32_t *cu, int32_t *lens_out, int32_t *free_count_out,
                               int32_t *status, cudaStream_t st)
{
    const ReserveParams prm{new_lens, lens, free_pages, free_count, block_table, slots, positions, cu, lens_out,
                            free_count_out, status, num_pages, T, B, page_shift, max_pages};
    // a CTA for each two tokens per thread, up to the portable cluster size
    int ctas = 1;
    while (ctas < 8 && static_cast<int64_t>(ctas) * kThreads * 2 < T) ctas *= 2;
    const size_t smem = sizeof(int32_t) * (3 * static_cast<size_t>(B) + 2);
    if (ctas == 1) {  // a cluster of its own
        reserve_kernel<<<1, kThreads, smem, st>>>(prm);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, reserve_kernel, prm);
}

cudaError_t launch_kv4_release(const int32_t *done, int32_t *lens, int B, int page_shift, int32_t *block_table,
                               int max_pages, int32_t *free_pages, int32_t *free_count, int64_t num_pages,
                               int32_t *status, cudaStream_t st)
{
    const ReleaseParams prm{done, lens, block_table, free_pages, free_count, status, num_pages, B, page_shift, max_pages};
    release_kernel<<<1, kThreads, sizeof(int32_t) * (static_cast<size_t>(B) + 1), st>>>(prm);
    return cudaGetLastError();
}

}  // namespace awq
