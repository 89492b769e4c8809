// read.cu -- cache slots read back as bf16 rows: the inverse of the append.
//
// Row i of the outputs is cache slot slot_mapping[i]: K and V as bf16, or code (times the
// scale of the slot's block and head), for keys plus k_ref, formed in float32 and rounded
// once to bf16.
//
// A gather bound by HBM: a warp a row of both tensors, a lane 8 elements at a time (8 or 16
// bytes in, 16 out), kUnroll such pieces in flight (eight: 9.6 us for 8.4).  Where rows are few
// several warps share one (500 E4M3 rows of 8 x 128: 2.7 us, 3.5 with a warp each).  14,449 INT8
// rows of 4 x 128 take 8.4 to 9.5 us (69 to 78% of a copy's rate; 61% of the issue slots, the rest waits
// for the slot and then for its rows), bf16 ones 8.8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace gqa {
namespace rd {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;
constexpr float kScaleFloor = 0x1p-64f;  // as the decode reads scales

struct Params {
    const uint8_t *k, *v;
    const float *ks, *vs, *k_ref;
    int scale_shift;
    const int64_t *slots;
    int64_t n, num_slots;
    KvPlace place;
    int head_shift, row_pieces;  // pieces of 8 elements: log2 of a head's, a row's
    int parts;  // warps of a row
    __nv_bfloat16 *k_out, *v_out;
    int32_t *err;
};

// Eight codes -> float32.
template <bool INT8>
__device__ __forceinline__ void widen(uint2 w, float (&x)[8]) {
    if constexpr (INT8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = (float)(int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = e4m3x2_to_f16x2((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

enum Fmt { kBF16 = 0, kE4M3 = 1, kINT8 = 2 };

template <int FMT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const Params p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    const int64_t head_stride = (p.place.rows == 0 ? 1 : p.place.rows) * (int64_t)p.place.head_bytes;
    for (int64_t it = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < p.n * p.parts;
         it += warps) {
        const int64_t row = p.parts == 1 ? it : it / p.parts;
        const int part = (int)(it - row * p.parts);
        const int64_t slot = __ldg(p.slots + row);
        const bool there = slot >= 0 && slot < p.num_slots;
        if (!there && lane == 0 && part == 0) report_error(p.err, ATTN_ERR_BOUNDS);
        const int64_t at = there ? p.place.head_offset(slot, 0) : 0;
        const int64_t scale_at = (there ? slot >> p.scale_shift : 0) * p.place.n_kv_heads;
        // pieces 0 .. row_pieces - 1 are K's, the others V's
        for (int i0 = part * 32 * kUnroll + lane; i0 < 2 * p.row_pieces;
             i0 += p.parts * 32 * kUnroll) {
            uint4 a[kUnroll];
            float s[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const bool is_v = i0 + 32 * u >= p.row_pieces;
                const int i = i0 + 32 * u - (is_v ? p.row_pieces : 0);
                const int h = i >> p.head_shift, piece = i & ((1 << p.head_shift) - 1);
                a[u] = make_uint4(0u, 0u, 0u, 0u);
                s[u] = 1.f;
                if (i >= p.row_pieces || !there) continue;
                const uint8_t *src = (is_v ? p.v : p.k) + at + h * head_stride;
                if constexpr (FMT == kBF16) {
                    a[u] = __ldg(reinterpret_cast<const uint4 *>(src) + piece);
                } else {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(src) + piece);
                    a[u].x = w.x, a[u].y = w.y;
                    const float *scales = is_v ? p.vs : p.ks;
                    if (scales != nullptr) s[u] = fmaxf(__ldg(scales + scale_at + h), kScaleFloor);
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const bool is_v = i0 + 32 * u >= p.row_pieces;
                const int i = i0 + 32 * u - (is_v ? p.row_pieces : 0);
                if (i >= p.row_pieces) continue;
                if constexpr (FMT != kBF16) {
                    float x[8];
                    widen<FMT == kINT8>(make_uint2(a[u].x, a[u].y), x);
                    if (!is_v && p.k_ref != nullptr && there) {
                        const float4 r0 = __ldg(reinterpret_cast<const float4 *>(p.k_ref) + 2 * i);
                        const float4 r1 = __ldg(reinterpret_cast<const float4 *>(p.k_ref) + 2 * i + 1);
                        const float r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], s[u], r[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] *= s[u];
                    }
                    a[u] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                      pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
                }
                reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out)[row * p.row_pieces + i] = a[u];
            }
        }
    }
}

}  // namespace rd

int launch_kv_read(const int64_t *slot_mapping, int64_t n, const attn_kv_cache *cache,
                   int n_kv_heads, int head_dim, void *k_out, void *v_out, int32_t *err,
                   cudaStream_t stream) {
    rd::Params p = {};
    const bool scaled = kv_scaled(cache->dtype);
    p.k = static_cast<const uint8_t *>(cache->k);
    p.v = static_cast<const uint8_t *>(cache->v);
    p.ks = scaled ? cache->k_scale : nullptr;
    p.vs = scaled ? cache->v_scale : nullptr;
    p.k_ref = cache->dtype == ATTN_KV_BF16 ? nullptr : cache->k_ref;
    if (scaled)
        while ((1 << p.scale_shift) < cache->scale_block) ++p.scale_shift;
    p.slots = slot_mapping;
    p.n = n;
    p.num_slots = cache->num_slots;
    p.place = kv_place(cache, n_kv_heads, head_dim, cache->dtype == ATTN_KV_BF16 ? 2 : 1);
    p.head_shift = head_dim == 128 ? 4 : 3;
    p.row_pieces = n_kv_heads << p.head_shift;
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    p.v_out = static_cast<__nv_bfloat16 *>(v_out);
    p.err = err;
    const int per_block = rd::kThreads / 32;
    const int64_t cap = (int64_t)device_sm_count() * 16;
    // few rows: a warp for each kUnroll pieces a lane
    const int64_t most = (2 * (int64_t)p.row_pieces + 32 * rd::kUnroll - 1) / (32 * rd::kUnroll);
    p.parts = (int)std::max<int64_t>(1, std::min<int64_t>(most, cap * per_block / n));
    int64_t blocks = (n * p.parts + per_block - 1) / per_block;
    if (blocks > cap) blocks = cap;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)blocks), dim3(rd::kThreads), 0, stream, p);
    };
    const cudaError_t e = cache->dtype == ATTN_KV_BF16          ? go(rd::kv_read_kernel<rd::kBF16>)
                          : cache->dtype == ATTN_KV_INT8_SCALED ? go(rd::kv_read_kernel<rd::kINT8>)
                                                                : go(rd::kv_read_kernel<rd::kE4M3>);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace gqa
