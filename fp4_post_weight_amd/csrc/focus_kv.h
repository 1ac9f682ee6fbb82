// focus_kv.h -- arguments, device helpers and launchers of the paged 8-bit
// cache of keys and values (write, read back, attention), shared by
// focus_kv.hip, focus_attention.hip and the C ABI.  Arguments reaching the
// launchers have been validated on the host.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace focus {

struct KvCacheArgs {
    uint8_t *kc, *ks;  // [pages, kv_heads, page, dim], [pages, kv_heads]
    uint8_t *vc, *vs;  // [pages, kv_heads, dim, page], [pages, kv_heads]
    int pages, kv_heads;
    int dim;           // 64 or 128
    int log_page;      // 4..7
};

struct KvBatchArgs {
    const int* table;  // [sequences] rows of max_pages, table_stride apart
    int64_t table_stride;
    int max_pages;
    const int* lengths;
    const int* cu;     // [sequences + 1] or NULL: one row per sequence
    int sequences;
    int tokens;
};

// Angles' cosines and sines [positions, dim] (cosines first), or NULL.
struct RopeArgs {
    const float* table;
    int64_t positions;
};

struct KvAttentionArgs {
    KvCacheArgs cache;
    KvBatchArgs batch;
    RopeArgs rope;
    const uint16_t* q;  // rows of heads * dim BF16, q_stride elements apart
    int64_t q_stride;
    int heads;
    float scale, softcap;
    int window;         // 0: none
    uint16_t* y;        // [tokens, heads * dim] BF16
    float* workspace;
    int64_t workspace_bytes;
};

hipError_t launch_rope_table(const double* inv_freq, int64_t positions, int64_t dim, float* table, hipStream_t stream);

hipError_t launch_kv_write(const KvCacheArgs& c, const KvBatchArgs& b, const RopeArgs& r, const uint16_t* k,
                           int64_t k_stride, const uint16_t* v, int64_t v_stride, hipStream_t stream);

hipError_t launch_kv_read(const KvCacheArgs& c, const KvBatchArgs& b, uint16_t* k, uint16_t* v, hipStream_t stream);

// Whether the launches stay within 2^32 threads.
bool kv_pages_fit(const KvCacheArgs& c, const KvBatchArgs& b);
bool kv_attention_fits(const KvCacheArgs& c, const KvBatchArgs& b, int heads);

hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t stream);

// Bytes for the largest split of launch_kv_attention.
int64_t kv_attention_workspace_bytes(const KvCacheArgs& c, const KvBatchArgs& b, int heads);

#if defined(__HIP__)

// A sequence's rows in the step's tensors and its tokens in the cache.  Values
// outside the tensors (the arrays are device memory, never checked on the host)
// are brought into range, so that no later access leaves them.
struct KvSequence {
    int row0, rows;
    int64_t length;
    __device__ __forceinline__ int64_t first() const { return length - rows; }  // position of row 0, may be negative
};

__device__ __forceinline__ int kv_row_at(const KvBatchArgs& b, int i) { return min(max(b.cu[i], 0), b.tokens); }

__device__ __forceinline__ KvSequence kv_sequence(const KvBatchArgs& b, int i) {
    KvSequence s;
    s.row0 = i;
    s.rows = 1;
    if (b.cu) {
        s.row0 = kv_row_at(b, i);
        s.rows = max(kv_row_at(b, i + 1) - s.row0, 0);
    }
    s.length = max(b.lengths[i], 0);
    return s;
}

// Pages of ragged sequences without a count of them on the host: sequence i
// owns the items from (cu[i] >> log_page) + 2 i on, at least as many as the
// pages that its rows can touch.  Returns the sequence of an item and its number
// in it; items that a sequence does not need lie behind its last page.  Every
// wavefront of the workgroup calls it, all 64 lanes.
__device__ __forceinline__ int kv_find(const KvBatchArgs& b, int log_page, int item, int& number) {
    if (!b.cu) {
        number = 0;
        return item;
    }
    const int lane = threadIdx.x & 63;
    int count = 0;  // sequences that begin at or before the item
    for (int base = 0; base < b.sequences; base += 64) {
        const int i = base + lane;
        const bool before = i < b.sequences && (kv_row_at(b, i) >> log_page) + 2 * i <= item;
        count += __popcll(__ballot(before));
    }
    const int i = max(count - 1, 0);
    number = item - ((kv_row_at(b, i) >> log_page) + 2 * i);
    return i;
}

#endif

// How many items kv_find can be asked for.
inline int64_t kv_items(const KvBatchArgs& b, int log_page) {
    return b.cu ? ((int64_t)b.tokens >> log_page) + 2 * (int64_t)b.sequences : b.sequences;
}

}  // namespace focus
