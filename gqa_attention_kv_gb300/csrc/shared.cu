// shared.cu -- decode attention for a batch whose requests share prefixes.
//
// What is computed: attn_decode's softmax over the visible keys of each row, where key t of
// request b lies in its own slots for t >= prefix_lens[b] and in those of row
// prefix_rows[b] before.  The plainest form: a warp a query row and head, a running maximum
// and sum in float32, every key read by every row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace gqa {
namespace shr {

enum Fmt { kBF16 = 0, kE4M3 = 1, kINT8 = 2 };

struct Params {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    const uint8_t *k, *v;
    const float *ks, *vs;
    int scale_shift;
    int kind, slots_per_seq, block_size, max_blocks, num_pages, n_rows;
    KvPlace place;
    const int32_t *block_table, *seq_lens, *positions, *prefix_rows, *prefix_lens;
    int batch, q_rows, n_q_heads, n_kv_heads, group, window, max_seq_len, max_prefix_len;
    float scale_log2;
    int32_t *err;
};

template <int FMT, int HD>
__global__ void __launch_bounds__(128) shared_simple_kernel(const Params p) {
    constexpr int V = HD / 32;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (i >= (int64_t)p.batch * p.q_rows * p.n_q_heads) return;
    const int h = (int)(i % p.n_q_heads), kvh = h / p.group;
    const int64_t row = i / p.n_q_heads;
    const int b = (int)(row / p.q_rows);
    int len = p.seq_lens[b];
    const int cap = p.kind == ATTN_CACHE_LINEAR ? min(p.max_seq_len, p.slots_per_seq) : p.max_seq_len;
    if (len < 0 || len > cap) {
        report_error(p.err, ATTN_ERR_BOUNDS);
        len = max(0, min(len, cap));
    }
    int plen = p.prefix_lens[b], prow = 0;
    if (plen < 0 || plen > p.max_prefix_len) {
        report_error(p.err, ATTN_ERR_BOUNDS);
        plen = max(0, min(plen, p.max_prefix_len));
    }
    bool good = true;
    if (plen > 0) {
        prow = p.prefix_rows[b];
        good = prow >= 0 && prow < p.n_rows;
        if (!good) report_error(p.err, ATTN_ERR_BOUNDS);
    }
    const int pos = p.positions[row];
    const int hi = min(len, pos + 1), lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    float q[V], o[V] = {}, m = -INFINITY, l = 0.f;
    for (int d = 0; d < V; ++d) q[d] = __bfloat162float(p.q[i * HD + lane * V + d]);
    for (int t = lo; t < hi; ++t) {
        const bool pre = t < plen;
        if (pre && !good) continue;
        const int r = pre ? prow : b;
        int64_t slot;
        if (p.kind == ATTN_CACHE_PAGED) {
            const int page = p.block_table[(int64_t)r * p.max_blocks + t / p.block_size];
            if (page < 0 || page >= p.num_pages) {
                report_error(p.err, ATTN_ERR_BOUNDS);
                continue;
            }
            slot = (int64_t)page * p.block_size + t % p.block_size;
        } else {
            slot = (int64_t)r * p.slots_per_seq + t;
        }
        const int64_t at = p.place.head_offset(slot, kvh);
        float k[V], v[V];
        for (int d = 0; d < V; ++d) {
            const int e = lane * V + d;
            if constexpr (FMT == kBF16) {
                k[d] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.k + at)[e]);
                v[d] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.v + at)[e]);
            } else if constexpr (FMT == kINT8) {
                k[d] = (float)(int8_t)p.k[at + e];
                v[d] = (float)(int8_t)p.v[at + e];
            } else {
                const uint32_t w = e4m3x2_to_f16x2(p.k[at + e] | (uint32_t)p.v[at + e] << 8);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                k[d] = f.x;
                v[d] = f.y;
            }
        }
        float s = 0.f, ks = 1.f, vs = 1.f;
        for (int d = 0; d < V; ++d) s = fmaf(q[d], k[d], s);
        for (int o2 = 16; o2 > 0; o2 >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o2);
        if (p.ks != nullptr) {
            ks = fmaxf(p.ks[(slot >> p.scale_shift) * p.n_kv_heads + kvh], 0x1p-64f);
            vs = fmaxf(p.vs[(slot >> p.scale_shift) * p.n_kv_heads + kvh], 0x1p-64f);
        }
        s *= ks * p.scale_log2;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
        m = mn;
        l = l * f + w;
        for (int d = 0; d < V; ++d) o[d] = o[d] * f + w * vs * v[d];
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int d = 0; d < V; ++d) p.out[i * HD + lane * V + d] = __float2bfloat16(o[d] * inv);
}

}  // namespace shr

int plan_shared(const attn_kv_cache *cache, int batch, int q_rows, int n_q_heads, int n_kv_heads,
                int head_dim, int max_seq_len, int max_prefix_len, int window, SharedPlan *plan) {
    plan->workspace = 256;
    return ATTN_OK;
}

int launch_shared(const SharedPlan &plan, const void *q, const attn_kv_cache *cache, int n_rows,
                  const int32_t *seq_lens, const int32_t *positions, const int32_t *prefix_rows,
                  const int32_t *prefix_lens, int batch, int q_rows, int max_seq_len,
                  int max_prefix_len, int window, int n_q_heads, int n_kv_heads, int head_dim,
                  float scale, void *out, void *workspace, int32_t *err, cudaStream_t stream) {
    shr::Params p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.k = static_cast<const uint8_t *>(cache->k);
    p.v = static_cast<const uint8_t *>(cache->v);
    const bool scaled = kv_scaled(cache->dtype);
    p.ks = scaled ? cache->k_scale : nullptr;
    p.vs = scaled ? cache->v_scale : nullptr;
    if (scaled)
        while ((1 << p.scale_shift) < cache->scale_block) ++p.scale_shift;
    p.kind = cache->kind;
    p.slots_per_seq = cache->slots_per_seq;
    p.block_size = cache->block_size;
    p.max_blocks = cache->max_blocks_per_seq;
    p.num_pages = cache->kind == ATTN_CACHE_PAGED ? (int)(cache->num_slots / cache->block_size) : 0;
    p.n_rows = n_rows;
    p.place = kv_place(cache, n_kv_heads, head_dim, cache->dtype == ATTN_KV_BF16 ? 2 : 1);
    p.block_table = cache->block_table;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.prefix_rows = prefix_rows;
    p.prefix_lens = prefix_lens;
    p.batch = batch;
    p.q_rows = q_rows;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = n_q_heads / n_kv_heads;
    p.window = window;
    p.max_seq_len = max_seq_len;
    p.max_prefix_len = std::min(max_prefix_len,
                                cache->kind == ATTN_CACHE_LINEAR ? cache->slots_per_seq : max_seq_len);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err = err;
    const int64_t rows = (int64_t)batch * q_rows * n_q_heads;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, p);
    };
    cudaError_t e;
    if (cache->dtype == ATTN_KV_BF16)
        e = head_dim == 128 ? go(shr::shared_simple_kernel<shr::kBF16, 128>)
                            : go(shr::shared_simple_kernel<shr::kBF16, 64>);
    else if (cache->dtype == ATTN_KV_INT8_SCALED)
        e = head_dim == 128 ? go(shr::shared_simple_kernel<shr::kINT8, 128>)
                            : go(shr::shared_simple_kernel<shr::kINT8, 64>);
    else
        e = head_dim == 128 ? go(shr::shared_simple_kernel<shr::kE4M3, 128>)
                            : go(shr::shared_simple_kernel<shr::kE4M3, 64>);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace gqa
