// kv4.cuh -- the paged 4-bit key/value cache: layout and launchers (internal).
//
// A cache is [num_pages, kv_heads, page_size / 16] blocks.  A block holds 16
// tokens of one head, 16 D + 128 bytes (a multiple of 128):
//   [0, 8 D)          keys:   16 rows of D / 2 bytes, channel 8 w + j in bits
//                     [4 j, 4 j + 4) of the row's word w (as in Q)
//   [8 D, 16 D)       values, the same
//   [16 D, +64)       a word per token for its key: the step (binary16) in the
//                     low half, the zero point in the high half
//   [16 D + 64, +64)  the same for its value
// Keys and values of a token range, with their steps, are then one contiguous
// piece: the attention fetches it with one bulk copy per page.
#pragma once

#include "awq_common.cuh"

namespace awq {

constexpr int kKvBlock = 16;  // tokens per block

__host__ __device__ constexpr int kv4_block_bytes(int D) { return 16 * D + 128; }

// the cache of one layer
struct Kv4Cache {
    uint8_t *data;
    int64_t num_pages;
    int heads, D;
    int page_shift;  // log2(page_size), 4..8
};

struct Kv4Tables {
    const int32_t *block_table;  // [B, max_pages]
    const int32_t *lens;         // [B]
    const int32_t *cu;           // [B + 1], or NULL: one query per request
    int B, max_pages;
};

// kv4_pages.cu
cudaError_t configure_kv4_pages();
cudaError_t launch_kv4_reserve(const int32_t *new_lens, const int32_t *lens, int B, int page_shift,
                               int32_t *block_table, int max_pages, const int32_t *free_pages,
                               const int32_t *free_count, int64_t num_pages, int64_t T, int64_t *slots,
                               int32_t *positions, int32_t *cu, int32_t *lens_out, int32_t *free_count_out,
                               int32_t *status, cudaStream_t st);
cudaError_t launch_kv4_release(const int32_t *done, int32_t *lens, int B, int page_shift, int32_t *block_table,
                               int max_pages, int32_t *free_pages, int32_t *free_count, int64_t num_pages,
                               int32_t *status, cudaStream_t st);

// kv4_store.cu
cudaError_t launch_kv4_append(const Kv4Cache &c, const __half *k, int64_t k_stride, const __half *v,
                              int64_t v_stride, const int64_t *slots, int64_t T, int32_t *status, cudaStream_t st);
cudaError_t launch_kv4_load(const Kv4Cache &c, const int64_t *slots, int64_t T, __half *k, __half *v,
                            int32_t *status, cudaStream_t st);

// kv4_attend.cu
struct Kv4AttendArgs {
    Kv4Cache cache;
    Kv4Tables tab;
    const __half *q;   // [T, q_stride], heads of D
    int64_t q_stride;
    __half *out;       // [T, q_heads, D]
    int64_t T;
    int max_new, q_heads, window;
    float scale;
    int32_t *status;
};
// Query rows (queries times heads of a group) of a request above which the prompt
// kernel takes it.  The split kernel covers 16 rows per pass over the cache, the
// prompt kernel 256, at a higher fixed cost.  Measured, split against prompt
// kernel, in us: 32 rows 39 / 47 (1 x 32000 keys), 47 / 77 (16 x 4000); 64 rows
// 57 / 49 and 156 / 100 (32 x 4000); 128 rows 94 / 51.
constexpr int kPromptRows = 48;
cudaError_t configure_kv4_attend();
// Whether the longest line of tiles that B requests of at most `rows` rows and `tokens` cached tokens can make
// is counted in 32 bits.
bool kv4_attend_countable(int64_t B, int64_t heads, int64_t rows, int64_t tokens);
size_t kv4_attend_workspace(int D);
// requests with more than max_rows rows are left to the prompt kernel
cudaError_t launch_kv4_attend(const Kv4AttendArgs &a, int64_t max_rows, void *ws, int num_sms, cudaStream_t st);

// kv4_prefill.cu -- the requests with more than kPromptRows rows: tcgen05
cudaError_t configure_kv4_prefill();
size_t kv4_prefill_workspace(int D);
cudaError_t launch_kv4_prefill(const Kv4AttendArgs &a, void *ws, int num_sms, cudaStream_t st);

}  // namespace awq
