// kernels.h -- host-side launchers shared between the C ABI and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/attn_kv.h"

namespace gqa {

int device_sm_count();

// The last CUDA runtime error a launch in this thread ran into (cudaSuccess if
// none); attn_last_cuda_error() reports it to the caller.
void note_cuda_error(cudaError_t e);

// Launch with programmatic stream serialisation: the kernel may begin while
// its predecessor on the stream finishes; it must call pdl_wait() before
// touching memory the predecessor writes.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<Args &&>(args)...);
    if (e != cudaSuccess) note_cuda_error(e);
    return e;
}

// Encode a 2D/3D tensor map of bf16 (or, with bytes, 8-bit) elements, with
// 128-byte swizzle (returns false on failure).
bool encode_tensor_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims,
                       const uint64_t *strides_bytes, const uint32_t *box, bool swizzle128,
                       bool bytes = false);
// The same over f16 elements, 128-byte swizzled (boxes of 64 columns).
bool encode_tensor_map_f16(CUtensorMap *map, const void *base, int rank, const uint64_t *dims,
                           const uint64_t *strides_bytes, const uint32_t *box);

// Where head h's row of cache slot s starts, in bytes (attn_kv_cache's layouts):
// slot-major (rows == 0) or head-major inside blocks of `rows` slots.
struct KvPlace {
    int64_t rows;    // 0: ATTN_LAYOUT_BSHD; else the block size of ATTN_LAYOUT_BHSD
    int n_kv_heads;
    int head_bytes;  // head_dim x element size
    __host__ __device__ __forceinline__ int64_t head_offset(int64_t s, int h) const {
        return rows == 0 ? (s * n_kv_heads + h) * head_bytes
                         : (((s / rows) * n_kv_heads + h) * rows + s % rows) * head_bytes;
    }
};

// The placement a cache descriptor asks for (element size esize bytes).
inline KvPlace kv_place(const attn_kv_cache *c, int n_kv_heads, int head_dim, int esize) {
    KvPlace p;
    p.rows = c->layout == ATTN_LAYOUT_BHSD
                 ? (c->kind == ATTN_CACHE_PAGED ? c->block_size : c->slots_per_seq)
                 : 0;
    p.n_kv_heads = n_kv_heads;
    p.head_bytes = head_dim * esize;
    return p;
}

int launch_kv_append(const void *k_new, const void *v_new, const int64_t *slot_mapping, int64_t n,
                     void *k_cache, void *v_cache, int64_t num_slots, const KvPlace &place,
                     int32_t *err, cudaStream_t stream);

// FP8 cache append: row_elems = n_kv_heads * head_dim (a multiple of 16);
// k_ref float32 [row_elems] or nullptr.
int launch_kv_append_fp8(const void *k_new, const void *v_new, const float *k_ref,
                         const int64_t *slot_mapping, int64_t n, void *k_cache, void *v_cache,
                         int64_t num_slots, const KvPlace &place, int32_t *err,
                         cudaStream_t stream);

// ref[e] = mean over n rows of the bf16 matrix k[n][row_elems], as float32.
int launch_kv_reference(const void *k, int64_t n, int row_elems, float *ref,
                        cudaStream_t stream);

// Chunk plan (many query rows per KV group over a linear slot-major bf16
// cache, chunk.cu): rt chunk rows per 128-row tcgen05 tile, n_pairs tile
// pairs, n_split CTAs along each key range, and the partial states (n_split >
// 1: f16 O, fp32 log-sum-exp) the merge combines.
struct ChunkPlan {
    int rt, n_pairs, n_split;
    size_t workspace;
};

void plan_chunk(int batch, int q_rows, int n_q_heads, int n_kv_heads, int head_dim,
                int max_seq_len, int window, ChunkPlan *plan);

// k_new / v_new / slot_mapping non-null: the step's rows are taken from
// k_new / v_new and written to the cache by the same launch (attn_decode_append).
int launch_chunk(const ChunkPlan &plan, const void *q, const attn_kv_cache *cache,
                 const int32_t *seq_lens, const int32_t *positions, int batch, int q_rows,
                 int max_seq_len, int window, int n_q_heads, int n_kv_heads, int head_dim,
                 float scale, void *out, void *workspace, int32_t *err, cudaStream_t stream,
                 const void *k_new = nullptr, const void *v_new = nullptr,
                 const int64_t *slot_mapping = nullptr);

// Decode plan: a persistent grid of one CTA per SM; requests are processed
// in launches of at most batch_per_launch (the per-request tables live in
// shared memory).
struct DecodePlan {
    int head_dim;
    int m_tiles;          // 0: <= 8 rows per unit (keys as MMA rows); 1, 2: 16-row tiles
    int rows;             // q_rows * group
    int row_blocks;       // units along the query rows of one KV head
    int grid;             // CTAs of the split kernel
    int batch_per_launch;
    size_t workspace;     // bytes of scratch: merge counters + fp32 partial states
    size_t counter_offset, counter_bytes;  // the counters, which must be zero between calls
    size_t partial_offset;                 // the partial states (after the counters)
    bool merge_kernel;    // units spanning very many CTAs are merged by a second kernel
    // Many rows per KV group over a linear slot-major bf16 cache go to the
    // tcgen05 chunk kernel instead (not with a fused rotary embedding, which
    // stays on the split kernel: the workspace covers both).
    bool chunk;
    ChunkPlan cp;
    size_t chunk_offset;  // the chunk's partial states, after the split kernel's scratch
};

int plan_decode(const attn_kv_cache *cache, int batch, int q_rows, int n_q_heads, int n_kv_heads,
                int head_dim, int max_seq_len, int window, DecodePlan *plan);

// Every host-side check attn_decode makes before it looks at the workspace;
// on success (and batch > 0) fills *plan.  Returns the attn_status.
int validate_decode(const void *q, const attn_kv_cache *cache, const int32_t *seq_lens,
                    const int32_t *positions, int batch, int q_rows, int max_seq_len, int window,
                    int n_q_heads, int n_kv_heads, int head_dim, float scale, const void *out,
                    DecodePlan *plan);

// k_new / v_new / slot_mapping non-null: the step's rows are appended by the
// same launch (attn_decode_append).
int launch_decode(const DecodePlan &plan, const void *q, const attn_kv_cache *cache,
                  const int32_t *seq_lens, const int32_t *positions, int batch, int q_rows,
                  int max_seq_len, int window, int n_q_heads, int n_kv_heads, float scale,
                  void *out, void *workspace, int32_t *err, cudaStream_t stream,
                  const void *k_new = nullptr, const void *v_new = nullptr,
                  const int64_t *slot_mapping = nullptr, const float *rope_inv_freq = nullptr,
                  bool tables_early = false, bool cache_early = false);

// Whether a cache's elements are 8-bit codes with a scale per block and head.
inline bool kv_scaled(int dtype) {
    return dtype == ATTN_KV_FP8_E4M3_SCALED || dtype == ATTN_KV_INT8_SCALED;
}

// Append to a scaled cache (scale_block slots and a head share a scale).
int launch_kv_append_scaled(const void *k_new, const void *v_new, const int64_t *slot_mapping,
                            int64_t n, const attn_kv_cache *cache, int n_kv_heads, int head_dim,
                            int32_t *err, cudaStream_t stream);

// Plan of attend.cu's decode: scaled caches, and any cache under a sliding window
// with sinks.  (request, row block) pairs go to the
// kernel per_launch at a time.
struct AttendPlan {
    int mt;     // 0: up to 8 rows per unit, 1: 16
    int heads;  // KV heads of a unit
    int row_blocks, entries, per_launch, grid, launches;
    int pieces;  // shares that the work of a launch is cut into
    bool merge;  // the parts of a unit are added up by a second kernel
    size_t count_offset, parts_offset, lse_offset, o_offset, workspace;
};

// ATTN_OK, or ATTN_ERR_SHAPE for sizes past the kernel's index range.  parts: for
// launch_attend_parts.
int plan_attend(const attn_kv_cache *cache, int batch, int q_rows, int n_q_heads, int n_kv_heads,
                int head_dim, int max_seq_len, int window, int sinks, AttendPlan *plan,
                bool parts = false);

int launch_attend(const AttendPlan &plan, const void *q, const attn_kv_cache *cache,
                  const int32_t *seq_lens, const int32_t *positions, int q_rows, int max_seq_len,
                  int window, int sinks, int n_q_heads, int n_kv_heads, int head_dim, float scale,
                  void *out, void *workspace, int32_t *err, cudaStream_t stream);

// What attend.cu leaves of keys at and behind a position of each request: partial states
// for a merge of the caller's (unit = (entry, KV heads together), see attend_merge_kernel).
struct AttendParts {
    const float *o, *lse;
    const int2 *parts;  // per unit: first and last (less than the first: none)
    int32_t *next;      // the launch's counter of shares, to be left at 0
    int rb, heads, row_blocks, e0, n_entries;
    float held;  // lse holds log2 of the sum of weights times 2^held
};

// One launch of the plan, its entries from e0 on, over keys t >= from[b] (clipped to
// 0 .. from_cap).  late_wait: what the stream's launch before this one writes after letting it
// begin is not read by this one (but by whoever merges the parts), and that launch waited for
// everything before it.  The first of the workspace's counters (0 between calls) counts the shares;
// whoever merges the parts sets it to 0 again.
int launch_attend_parts(const AttendPlan &plan, int e0, const int32_t *from, int from_cap,
                        const void *q, const attn_kv_cache *cache, const int32_t *seq_lens,
                        const int32_t *positions, int q_rows, int max_seq_len, int window,
                        int n_q_heads, int n_kv_heads, int head_dim, float scale, void *out,
                        void *workspace, int32_t *err, cudaStream_t stream, bool late_wait,
                        AttendParts *parts);

// Norms and rotary embedding of q and k (rope.cu); cache null: none is written to.
int launch_qk_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                   int64_t v_stride, const int32_t *positions, const int64_t *slot_mapping,
                   int64_t n, const attn_rope *r, const attn_kv_cache *cache, int n_q_heads,
                   int n_kv_heads, int head_dim, void *q_out, void *k_out, int32_t *err,
                   cudaStream_t stream);

// Cache slots as bf16 rows (read.cu).
int launch_kv_read(const int64_t *slot_mapping, int64_t n, const attn_kv_cache *cache,
                   int n_kv_heads, int head_dim, void *k_out, void *v_out, int32_t *err,
                   cudaStream_t stream);

// Decode with shared prefixes (shared.cu).
struct SharedPlan {
    AttendPlan own;  // of the keys that are not shared
    size_t rows_offset, lse_offset, o_offset, workspace;
};

int plan_shared(const attn_kv_cache *cache, int batch, int q_rows, int n_q_heads, int n_kv_heads,
                int head_dim, int max_seq_len, int window, SharedPlan *plan);

int launch_shared(const SharedPlan &plan, const void *q, const attn_kv_cache *cache, int n_rows,
                  const int32_t *seq_lens, const int32_t *positions, const int32_t *prefix_rows,
                  const int32_t *prefix_lens, int batch, int q_rows, int max_seq_len,
                  int max_prefix_len, int window, int n_q_heads, int n_kv_heads, int head_dim,
                  float scale, void *out, void *workspace, int32_t *err, cudaStream_t stream);

// Page operations (pages.cu).
int launch_pages_free(int32_t *block_table, int max_blocks, int table_rows, const int32_t *rows,
                      const int32_t *from_block, const int32_t *to_block, int n, int32_t *refs,
                      int num_pages, int32_t *err, cudaStream_t stream);
int launch_pages_reserve(int32_t *block_table, int max_blocks, int table_rows,
                         const int32_t *rows, const int32_t *from_block, const int32_t *to_block,
                         int n, int32_t *refs, int num_pages, int32_t *err, cudaStream_t stream);
int launch_pages_fork(int32_t *block_table, int max_blocks, int table_rows,
                      const int32_t *src_rows, const int32_t *dst_rows, const int32_t *seq_lens,
                      int n, int block_size, int32_t *refs, int num_pages, int32_t *moves,
                      int32_t *n_moves, int32_t *err, cudaStream_t stream);
size_t pages_workspace(int num_pages);
int launch_pages_compact(int32_t *block_table, int max_blocks, int table_rows, int block_size,
                         int32_t *refs, int num_pages, int32_t *moves, int max_moves,
                         int32_t *n_moves, int32_t *used, void *workspace, int32_t *err,
                         cudaStream_t stream);
int launch_pages_copy(const attn_kv_cache *caches, int n_caches, int n_kv_heads, int head_dim,
                      const int32_t *moves, const int32_t *n_moves, int max_moves, int32_t *err,
                      cudaStream_t stream);

int launch_prefill(const void *q, const void *k, const void *v, int batch, int seq_len,
                   int window, int n_q_heads, int n_kv_heads, int head_dim, float scale,
                   void *out, int32_t *err, cudaStream_t stream, int sinks = 0);

}  // namespace gqa
