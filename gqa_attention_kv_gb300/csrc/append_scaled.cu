// append_scaled.cu -- KV append into a cache of 8-bit codes with one scale per
// block of tokens and head.
//
// For one (block, KV head) and the call's rows x in the block (K less k_ref):
//     a  = max |x| over the rows' finite elements
//     s' = max(s, a / qmax, 2^-64), s = 0 when the call writes the block's
//          first slot (the block starts anew)          qmax = 448 (E4M3), 127 (INT8)
//     c' = round(c * (s * r)),  r = 1 / s'             the block's earlier codes, when s' > s > 0
//     c  = round(x * r)                                the new rows
// r and s * r are rounded to float32.  E4M3 rounds the float32 product, to
// nearest even, saturating; INT8 the exact product (one fused multiply-add
// against 1.5 * 2^23 leaves the integer in the low bits).  Scales only grow
// while a block fills, so a code is never clipped by a later row.
//
// One warp owns a (run of rows of one block, head, tensor): the maximum, the
// block's earlier codes and the new codes are its own, so there is nothing to
// synchronise and no order to depend on.  The kernel is a copy with arithmetic
// (HBM-bound): a run of up to 16 rows of 128 (32 of 64) stays in registers
// between its maximum and its codes, so each row is read once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "kernels.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr float kScaleFloor = 5.421010862427522e-20f;  // 2^-64
constexpr int kPasses = 8;                             // row groups held in registers

struct ScaledParams {
    const uint4 *k_new, *v_new;
    const float *k_ref;
    const int64_t *slots;
    int64_t n;
    uint8_t *k, *v;
    float *ks, *vs;
    int64_t num_slots;
    int shift;  // log2 of the slots of a block
    int window;  // rows a warp looks for run starts in
    KvPlace place;
    int32_t *err;
};

// The code of the exact product x * r, |x * r| < 2^21, as a byte.
template <bool CLAMP>
__device__ __forceinline__ uint32_t int8_code(float x, float r) {
    const float big = 12582912.f;  // 1.5 * 2^23
    float t = fmaf(x, r, big);
    if constexpr (CLAMP) t = fminf(fmaxf(t, big - 127.f), big + 127.f);
    return __float_as_uint(t);
}

// The larger of each half, NaN if either is.
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Codes of four values.
template <bool INT8, bool CLAMP = true>
__device__ __forceinline__ uint32_t encode4(const float *x, float r) {
    if constexpr (INT8) {
        const uint32_t a = int8_code<CLAMP>(x[0], r), b = int8_code<CLAMP>(x[1], r);
        const uint32_t c = int8_code<CLAMP>(x[2], r), d = int8_code<CLAMP>(x[3], r);
        return __byte_perm(__byte_perm(a, b, 0x0040u), __byte_perm(c, d, 0x0040u), 0x5410u);
    } else {
        return f32x2_to_e4m3x2(__fmul_rn(x[0], r), __fmul_rn(x[1], r)) |
               (f32x2_to_e4m3x2(__fmul_rn(x[2], r), __fmul_rn(x[3], r)) << 16);
    }
}

template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t w, float *x) {
    if constexpr (INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
    } else {
        const uint32_t lo = e4m3x2_to_f16x2(w), hi = e4m3x2_to_f16x2(w >> 16);
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(x[0]), "=f"(x[1])
            : "r"(lo));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(x[2]), "=f"(x[3])
            : "r"(hi));
    }
}

template <bool INT8, int HD>
__global__ void __launch_bounds__(128, 6) kv_append_scaled_kernel(const ScaledParams p) {
    constexpr int kLanes = HD / 8;           // lanes of a row: 16 bytes of bf16, 8 codes each
    constexpr int kRows = 32 / kLanes;       // rows of a pass
    constexpr float kQMax = INT8 ? 127.f : 448.f;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int heads = p.place.n_kv_heads;
    const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t group = warp / (2 * heads);
    const int rem = (int)(warp - group * (2 * heads)), tensor = rem / heads, h = rem - tensor * heads;
    const int64_t first_row = group * p.window;
    if (first_row >= p.n) return;
    const uint4 *src = tensor == 0 ? p.k_new : p.v_new;
    uint8_t *cache = tensor == 0 ? p.k : p.v;
    float *scales = tensor == 0 ? p.ks : p.vs;
    const float *ref = tensor == 0 && p.k_ref != nullptr
                           ? p.k_ref + h * HD + (lane & (kLanes - 1)) * 8
                           : nullptr;
    auto good = [&](int64_t s) { return s >= 0 && s < p.num_slots; };

    // Slots of rows first_row - 1 .. first_row + 30, a lane each, and the window's
    // rows themselves: nothing below waits for a second load where a run ends in
    // the window, as a prompt's do whose blocks begin with it.
    const int64_t seen = first_row - 1 + lane;
    const int64_t my_slot = seen >= 0 && seen < p.n ? __ldg(p.slots + seen) : -1;
    uint4 x[kPasses];
    auto fetch = [&](int64_t base, int64_t end, bool check) {
#pragma unroll
        for (int u = 0; u < kPasses; ++u) {
            const int64_t i = base + u * kRows + lane / kLanes;
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (i < end && (!check || good(__ldg(p.slots + i))))
                x[u] = __ldg(src + (i * heads + h) * kLanes + (lane & (kLanes - 1)));
        }
    };
    fetch(first_row, min(p.n, first_row + min(p.window, kPasses * kRows)), false);
    // rows of this window that start a run
    bool start = false;
    const int64_t before = __shfl_up_sync(0xffffffffu, my_slot, 1);
    if (lane >= 1 && lane <= p.window && seen < p.n) {
        if (good(my_slot)) {
            int64_t j = seen - 1, t = before;
            while (j >= 0 && !good(t))  // rows that are skipped do not end a run
                if (--j >= 0) t = __ldg(p.slots + j);
            start = j < 0 || (t >> p.shift) != (my_slot >> p.shift);
        } else if (rem == 0) {
            report_error(p.err, ATTN_ERR_BOUNDS);
        }
    }
    // the scales that the runs' blocks hold, all in one trip
    const float my_scale = start ? scales[(my_slot >> p.shift) * heads + h] : 0.f;
    uint32_t starts = __ballot_sync(0xffffffffu, start);
    bool intact = true;  // x holds the window's rows
    while (starts != 0) {
        const int at_lane = __ffs(starts) - 1;  // of the run's first row
        const int64_t i0 = first_row - 1 + at_lane;
        starts &= starts - 1;
        const int64_t block = __shfl_sync(0xffffffffu, my_slot, at_lane) >> p.shift;
        const int64_t inside = (int64_t(1) << p.shift) - 1;
        // the run: rows up to the first good slot of another block
        int64_t i1;
        bool fresh;
        {
            const bool in = seen < p.n && (!good(my_slot) || (my_slot >> p.shift) == block);
            const uint32_t out = ~__ballot_sync(0xffffffffu, in) & (0xffffffffu << at_lane);
            const int stop = out == 0 ? 32 : __ffs(out) - 1;
            i1 = first_row - 1 + stop;
            fresh = __any_sync(0xffffffffu, lane >= at_lane && lane < stop && good(my_slot) &&
                                                (my_slot & inside) == 0);
            while (i1 - (first_row - 1) >= 32 && i1 < p.n) {  // it goes on behind the 32 rows
                const int64_t i = i1 + lane;
                const int64_t s = i < p.n ? __ldg(p.slots + i) : 0;
                const uint32_t past = ~__ballot_sync(
                    0xffffffffu, i < p.n && (!good(s) || (s >> p.shift) == block));
                const int take = past == 0 ? 32 : __ffs(past) - 1;
                fresh |= __any_sync(0xffffffffu, lane < take && good(s) && (s & inside) == 0);
                i1 += take;
                if (take < 32) break;
            }
        }
        auto slot_of = [&](int64_t i) -> int64_t {  // all lanes together
            const int64_t l = i - (first_row - 1);
            const int64_t s = __shfl_sync(0xffffffffu, my_slot, (int)(l & 31));
            return l < 32 ? s : __ldg(p.slots + min(i, p.n - 1));
        };
        auto load = [&](int64_t base) { fetch(base, i1, true); };
        // the eight values of a lane's piece
        auto values = [&](const uint4 &w, float *f) {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[2 * e] = __uint_as_float(u[e] << 16);
                f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
            }
            if (ref != nullptr)
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __fsub_rn(f[e], __ldg(ref + e));
        };
        // The short way, a prompt's and a step's: the rows are in registers, in
        // consecutive slots, finite, and K has no reference.  Maxima are taken of bf16
        // pairs, INT8 codes need no clamp (|x r| <= 127 (1 + 2^-22)), addresses advance
        // by one stride.
        const int64_t slot0 = __shfl_sync(0xffffffffu, my_slot, at_lane);
        const int r0 = at_lane - 1;                                    // rows of the window
        const int r1 = (int)min(i1 - first_row, (int64_t)(kPasses * kRows + 1));
        const int my_r = lane / kLanes;  // this lane's row of the first pass
        bool short_way =
            intact && ref == nullptr && r1 <= min(p.window, kPasses * kRows) &&
            __all_sync(0xffffffffu, lane < at_lane || lane > r1 ||
                                        my_slot == slot0 + (lane - at_lane));
        float amax = 0.f;
        bool nan = false;
        if (short_way) {
            uint32_t mx = 0;
#pragma unroll
            for (int u = 0; u < kPasses; ++u) {
                if (my_r + u * kRows < r0 || my_r + u * kRows >= r1) continue;  // another run's
                mx = max_nan_bf16x2(mx, x[u].x & 0x7FFF7FFFu);
                mx = max_nan_bf16x2(mx, x[u].y & 0x7FFF7FFFu);
                mx = max_nan_bf16x2(mx, x[u].z & 0x7FFF7FFFu);
                mx = max_nan_bf16x2(mx, x[u].w & 0x7FFF7FFFu);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                mx = max_nan_bf16x2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float lo = __uint_as_float(mx << 16), hi = __uint_as_float(mx & 0xFFFF0000u);
            short_way = lo < INFINITY && hi < INFINITY;
            amax = fmaxf(lo, hi);
        }
        if (!short_way) {
        intact = false;
        amax = 0.f;
        for (int64_t base = i0; base < i1; base += kPasses * kRows) {
            load(base);
#pragma unroll
            for (int u = 0; u < kPasses; ++u) {
                const int64_t i = base + u * kRows + lane / kLanes, s = slot_of(i);
                if (i >= i1 || !good(s)) continue;
                float f[8];
                values(x[u], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = fabsf(f[e]);
                    nan |= a != a;
                    amax = fmaxf(amax, a < INFINITY ? a : 0.f);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        const int64_t at = block * heads + h;
        const float held = fresh ? 0.f : fmaxf(__shfl_sync(0xffffffffu, my_scale, at_lane), 0.f);
        const float now = fmaxf(fmaxf(held, __fdiv_rn(amax, kQMax)), kScaleFloor);
        const float r = __frcp_rn(now);
        if (!fresh && held > 0.f && now > held) {
            // the block's earlier codes under the new scale (the run's rows among them:
            // they are written below)
            const float by = __fmul_rn(held, r);
            constexpr int kL = HD / 16, kR = 32 / kL;  // 16 codes a lane
            for (int s0 = 0; s0 < (1 << p.shift); s0 += kR) {
                const int s = s0 + lane / kL;
                if (s >= (1 << p.shift)) continue;
                uint4 *c = reinterpret_cast<uint4 *>(
                    cache + p.place.head_offset((block << p.shift) + s, h) + (lane & (kL - 1)) * 16);
                uint4 w = *c;
                uint32_t *u = &w.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f[4];
                    decode4<INT8>(u[e], f);
                    u[e] = encode4<INT8>(f, by);
                }
                *c = w;
            }
        }
        __syncwarp();
        if (lane == 0) scales[at] = now;
        if (INT8 && __any_sync(0xffffffffu, nan)) {
            if (lane == 0) report_error(p.err, ATTN_ERR_UNSUPPORTED);
            nan = true;
        }
        if (short_way) {
            const int64_t row_bytes = (int64_t)p.place.head_bytes * (p.place.rows == 0 ? heads : 1);
            uint8_t *dst = cache + p.place.head_offset(slot0, h) + (my_r - r0) * row_bytes +
                           (lane & (kLanes - 1)) * 8;
#pragma unroll
            for (int u = 0; u < kPasses; ++u, dst += kRows * row_bytes) {
                if (my_r + u * kRows < r0 || my_r + u * kRows >= r1) continue;
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = __uint_as_float(w[e] << 16);
                    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
                }
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(encode4<INT8, false>(f, r), encode4<INT8, false>(f + 4, r));
            }
            __syncwarp();
            continue;
        }
        const bool kept = i1 - i0 <= kPasses * kRows;
        for (int64_t base = i0; base < i1; base += kPasses * kRows) {
            if (!kept) load(base);
#pragma unroll
            for (int u = 0; u < kPasses; ++u) {
                const int64_t i = base + u * kRows + lane / kLanes, s = slot_of(i);
                if (i >= i1 || !good(s)) continue;
                float f[8];
                values(x[u], f);
                if (INT8 && nan)  // INT8 has no NaN: 0
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = f[e] == f[e] ? f[e] : 0.f;
                *reinterpret_cast<uint2 *>(cache + p.place.head_offset(s, h) +
                                           (lane & (kLanes - 1)) * 8) =
                    make_uint2(encode4<INT8>(f, r), encode4<INT8>(f + 4, r));
            }
        }
        __syncwarp();
    }
}

}  // namespace

int launch_kv_append_scaled(const void *k_new, const void *v_new, const int64_t *slot_mapping,
                            int64_t n, const attn_kv_cache *cache, int n_kv_heads, int head_dim,
                            int32_t *err, cudaStream_t stream) {
    if (n <= 0) return ATTN_OK;
    ScaledParams p = {};
    p.k_new = static_cast<const uint4 *>(k_new);
    p.v_new = static_cast<const uint4 *>(v_new);
    p.k_ref = cache->k_ref;
    p.slots = slot_mapping;
    p.n = n;
    p.k = static_cast<uint8_t *>(cache->k);
    p.v = static_cast<uint8_t *>(cache->v);
    p.ks = cache->k_scale;
    p.vs = cache->v_scale;
    p.num_slots = cache->num_slots;
    while ((1 << p.shift) < cache->scale_block) ++p.shift;
    p.place = kv_place(cache, n_kv_heads, head_dim, 1);
    p.err = err;
    // A step's rows mostly start runs of their own: a warp each.  A prompt's are runs
    // of whole blocks: a warp takes the starts among 16 rows.  Which of the two a call
    // is shows in n alone, so a warp takes the fewest rows with which the warps are no
    // more than 64 an SM.
    const int64_t per_row = 2ll * n_kv_heads;
    p.window = 1;
    while (p.window < 16 && (n + p.window - 1) / p.window * per_row > (int64_t)device_sm_count() * 64)
        p.window *= 2;
    const int64_t warps = (n + p.window - 1) / p.window * per_row;
    const int64_t blocks = (warps + 3) / 4;
    if (blocks >= (int64_t(1) << 31)) return ATTN_ERR_SHAPE;
    const dim3 grid((unsigned)blocks), threads(128);
    cudaError_t e;
    if (cache->dtype == ATTN_KV_INT8_SCALED)
        e = head_dim == 128
                ? launch_pdl(kv_append_scaled_kernel<true, 128>, grid, threads, 0, stream, p)
                : launch_pdl(kv_append_scaled_kernel<true, 64>, grid, threads, 0, stream, p);
    else
        e = head_dim == 128
                ? launch_pdl(kv_append_scaled_kernel<false, 128>, grid, threads, 0, stream, p)
                : launch_pdl(kv_append_scaled_kernel<false, 64>, grid, threads, 0, stream, p);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace gqa
