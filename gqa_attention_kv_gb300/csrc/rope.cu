// rope.cu -- norms of queries and keys for each head and their rotary embedding in one
// pass, with the new keys and values written into the cache.
//
// What is computed, for a row x of one head (D dims) of a token at position p:
//     norm      x_d <- x_d w_d / sqrt(mean(x^2) + eps)         (where weights are given)
//     rotation  a_i = p inv_freq[i], c = factor cos a_i, s = factor sin a_i, i < rot / 2,
//               x1 <- x1 c - x2 s,  x2 <- x2 c + x1 s
//               with (x1, x2) = (x[2i], x[2i+1])  or  (x[i], x[i + rot/2]);
//               dims from rot on stay
// in float32, rounded once to bf16; keys for an E4M3 cache are then encoded from that bf16
// as attn_kv_append encodes them.  Values are copied (or encoded).
//
// Angles: a float32 product p inv_freq is off by p 2^-24 radians, a tenth of a turn's
// radian at a million tokens.  Only its fraction of a turn counts, so that is what is
// formed, in integers: F = inv_freq / (2 pi) as a 64-bit fraction of a turn (the mantissa
// times 2^64 / (2 pi), shifted), p F modulo 2^64 the fraction of p steps, and its upper 32
// bits, as a float of half turns, go to sincospif.  No 64-bit floating point (slow on this
// GPU) and no range reduction.
//
// GB300 mapping.  Every byte is read and written once: HBM bandwidth is the floor of a
// prompt, launch and load latency that of a step.  A lane holds 16 bytes of a head's row
// (16 lanes a row of 128 dims, 8 of 64), a warp takes two or four rows at a time and kUnroll
// such passes are in flight.  The token's sines and cosines are computed once a warp, two
// frequencies a lane, and go to the lanes that need them through shared memory; a pair
// whose halves lie in different lanes is exchanged by shuffles.  Where there are few tokens
// a token's heads are dealt to several warps (64 tokens of 32/8 x 128 with norms and append 4.1 us,
// a warp a token 11.9; 1,500 of 32/32 x 64 12.9 and 15.0; a prompt the same).
//
// Measured: 14,449 tokens of 28/4 x 128 44.7 us (5.29 TB/s, 78% of a copy's rate; 64% of the issue slots),
// with norms 55.7 (the sums of squares' shuffles and the factors of both weights: 71% of the issue
// slots), interleaved 44.2, appended to a linear cache 51.6 (bf16) or 52.2 (E4M3).  1,500 tokens of
// 32/32 x 64 with norms into a linear cache 12.8 (42% of a copy's rate): 56% of the issue slots at 17
// warps an SM; a warp asks for a round of rows and waits for it, three times, and V's rows, a third of
// them, go through the norm's sums and products to be written as they came.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace gqa {
namespace rope {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnroll = 4;  // passes (of two or four rows) whose loads are in flight
constexpr int kBlocks = 6;  // of an SM

// Where the halves of a pair stand
enum Mode {
    kPairs = 0,     // next to each other
    kHalves = 1,    // half of the rotated dims apart, whole 16-byte pieces
    kHalvesAny = 2  // ... any number of dims (through shared memory)
};

struct Params {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from a token's row to the next
    __nv_bfloat16 *q_out, *k_out;
    const int32_t *positions;
    const float *inv_freq, *q_weight, *k_weight;
    float factor, eps;
    int rot, n_q_heads, n_kv_heads, n_heads;  // n_heads: rows of a token, V's among them
    int64_t n;
    int chunks, chunk_passes;  // warps of a token, and the passes of each
    // cache (k_cache null: none)
    uint8_t *k_cache, *v_cache;
    const float *k_ref;
    const int64_t *slots;
    int64_t num_slots;
    KvPlace place;
    bool fp8;
    int32_t *err;
};

// inv_freq / (2 pi) modulo 1 as a 64-bit fraction.  m 2^(e - 23) / (2 pi) with a 24-bit m:
// m times floor(2^64 / (2 pi)) has 88 bits and is off by less than m, 2^(e + 1) units of
// 2^-64 after the shift.
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
    constexpr uint64_t kTurn = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
    const uint32_t w = __float_as_uint(inv_freq);
    const int e = (int)((w >> 23) & 255) - 127;
    const uint64_t m = (w & 0x7FFFFFu) | 0x800000u;
    if (e < -126) return 0;  // zero and subnormals
    const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
    const int s = 23 - e;
    uint64_t f;
    if (s >= 64)
        f = s >= 88 ? 0 : hi >> (s - 64);
    else if (s > 0)
        f = (lo >> s) | (hi << (64 - s));
    else
        f = s > -64 ? lo << -s : 0;
    return (w >> 31) ? 0 - f : f;
}

template <int HD, int MODE, bool NORM>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_kernel(const Params p) {
    constexpr int kLanes = HD / 8;         // lanes of a row
    constexpr int kRows = 32 / kLanes;     // rows of a pass
    __shared__ __align__(16) float2 turns[kWarps][HD / 2];  // cosine and sine of each frequency
    __shared__ __align__(16) float weights[NORM ? 2 : 1][NORM ? HD : 4];
    // Of queries and keys, for each dim what it and the other one of its pair are multiplied with
    // (turn and weight); dims d0 + 2 i and + 1 of all lanes stand together, or the lanes would
    // meet in four banks
    constexpr int kTypes = NORM ? 2 : 1;
    __shared__ float4 factors[kWarps][kTypes][4][kLanes];
    __shared__ float parked[MODE == kHalvesAny ? kWarps : 1][MODE == kHalvesAny ? kRows * HD : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / kLanes, piece = lane % kLanes, d0 = piece * 8;
    const int half = p.rot / 2;

    pdl_wait();
    pdl_launch_dependents();

    uint64_t step[HD / 64];  // of frequencies lane and lane + 32
#pragma unroll
    for (int i = 0; i < HD / 64; ++i)
        step[i] = lane + 32 * i < half ? turn_fraction(__ldg(p.inv_freq + lane + 32 * i)) : 0;
    if constexpr (NORM) {
        for (int i = threadIdx.x; i < HD; i += kThreads) {
            weights[0][i] = p.q_weight != nullptr ? __ldg(p.q_weight + i) : 1.f;
            weights[1][i] = p.k_weight != nullptr ? __ldg(p.k_weight + i) : 1.f;
        }
        __syncthreads();
    }
    // the lane that holds the other halves of this lane's pairs (kHalves)
    const int other = MODE != kHalves || d0 >= p.rot
                          ? lane
                          : sub * kLanes + (d0 < half ? piece + half / 8 : piece - half / 8);

    const int64_t items = p.n * p.chunks;
    for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < items;
         item += (int64_t)gridDim.x * kWarps) {
        const int64_t t = item / p.chunks;
        const int first = (int)(item - t * p.chunks) * p.chunk_passes * kRows;
        const int end = min(p.n_heads, first + p.chunk_passes * kRows);
        const int pos = __ldg(p.positions + t);
        const int64_t slot = p.slots != nullptr ? __ldg(p.slots + t) : 0;
        const bool stored = p.slots != nullptr && slot >= 0 && slot < p.num_slots;

        uint4 now[kUnroll];
        auto load = [&](int h0) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int h = h0 + u * kRows + sub;
                const __nv_bfloat16 *src =
                    h < p.n_q_heads                  ? p.q + t * p.q_stride + h * HD
                    : h < p.n_q_heads + p.n_kv_heads ? p.k + t * p.k_stride + (h - p.n_q_heads) * HD
                                                     : p.v + t * p.v_stride +
                                                           (h - p.n_q_heads - p.n_kv_heads) * HD;
                now[u] = make_uint4(0u, 0u, 0u, 0u);
                if (h < end) now[u] = __ldcs(reinterpret_cast<const uint4 *>(src + d0));
            }
        };
        load(first);  // (under way while the angles are computed)

        if (p.slots != nullptr && !stored && lane == 0 && first == 0)
            report_error(p.err, ATTN_ERR_BOUNDS);
        __syncwarp();  // the token before has been read
#pragma unroll
        for (int i = 0; i < HD / 64; ++i)
            if (lane + 32 * i < half) {
                const uint64_t f = (uint64_t)(int64_t)pos * step[i];
                float s, c;
                sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &s, &c);
                turns[warp][lane + 32 * i] = make_float2(c * p.factor, s * p.factor);
            }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) {
            const int d = lane + 32 * i;
            const bool low = MODE == kPairs ? !(d & 1) : d < half;
            const int pair = d >= p.rot ? d : MODE == kPairs ? d ^ 1 : low ? d + half : d - half;
            float2 turn = make_float2(1.f, 0.f);
            if (d < p.rot) turn = turns[warp][MODE == kPairs ? d / 2 : low ? d : d - half];
            if (low) turn.y = -turn.y;
#pragma unroll
            for (int t2 = 0; t2 < kTypes; ++t2) {
                float2 &f =
                    reinterpret_cast<float2 *>(&factors[warp][t2][(d & 7) >> 1][d >> 3])[d & 1];
                f = NORM ? make_float2(turn.x * weights[t2][d], turn.y * weights[t2][pair]) : turn;
            }
        }
        __syncwarp();
        float4 held[4];  // without norms one set serves all rows
        if constexpr (!NORM)
#pragma unroll
            for (int i = 0; i < 4; ++i) held[i] = factors[warp][0][i][piece];

        for (int h0 = first; h0 < end; h0 += kUnroll * kRows) {
            if (h0 != first) load(h0);
            float r[kUnroll];  // 1 / sqrt(mean square)
            if constexpr (NORM) {
                auto square_sums = [&](float by, float(&sum)[kUnroll]) {
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) {
                        const uint32_t raw[4] = {now[u].x, now[u].y, now[u].z, now[u].w};
                        sum[u] = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float a = __uint_as_float(raw[i] << 16) * by;
                            const float b = __uint_as_float(raw[i] & 0xFFFF0000u) * by;
                            sum[u] = fmaf(a, a, fmaf(b, b, sum[u]));
                        }
                    }
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
                        for (int u = 0; u < kUnroll; ++u)
                            sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
                };
                float sum[kUnroll];
                square_sums(1.f, sum);
                bool over = false;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    r[u] = rsqrtf(sum[u] * (1.f / HD) + p.eps);
                    over |= isinf(sum[u]);
                }
                // squares past float32: those of x 2^-64, beside which eps is nothing
                if (__any_sync(0xffffffffu, over)) {
                    float small[kUnroll];
                    square_sums(0x1p-64f, small);
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u)
                        if (isinf(sum[u])) r[u] = 0x1p-64f * rsqrtf(small[u] * (1.f / HD));
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (h0 + u * kRows >= end) break;
                const int h = h0 + u * kRows + sub;
                const bool is_q = h < p.n_q_heads, is_v = h >= p.n_q_heads + p.n_kv_heads;
                const uint32_t raw[4] = {now[u].x, now[u].y, now[u].z, now[u].w};
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = __uint_as_float(raw[i] << 16);
                    x[2 * i + 1] = __uint_as_float(raw[i] & 0xFFFF0000u);
                }
                float z[8];  // the others of the pairs
                if constexpr (MODE == kPairs) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[i] = x[i ^ 1];
                } else if constexpr (MODE == kHalves) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = __shfl_sync(0xffffffffu, raw[i], other);
                        z[2 * i] = __uint_as_float(w << 16);
                        z[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
                    }
                } else {
                    float *row = parked[warp] + sub * HD;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) row[d0 + i] = x[i];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int d = d0 + i;
                        z[i] = d < p.rot ? row[d < half ? d + half : d - half] : 0.f;
                    }
                }
                float y[8];
                const float by =
                    NORM && (is_q ? p.q_weight : p.k_weight) != nullptr ? r[u] : 1.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 g = NORM ? factors[warp][is_q ? 0 : kTypes - 1][i][piece] : held[i];
                    const int d = d0 + 2 * i;
                    // whole pieces turn or stay, but for odd numbers of dims
                    const bool on0 = MODE == kHalves ? d0 < p.rot : d < p.rot;
                    const bool on1 = MODE == kHalves ? d0 < p.rot : d + 1 < p.rot;
                    const float a = NORM ? x[2 * i] * by : x[2 * i];
                    const float b = NORM ? x[2 * i + 1] * by : x[2 * i + 1];
                    const float za = NORM ? z[2 * i] * by : z[2 * i];
                    const float zb = NORM ? z[2 * i + 1] * by : z[2 * i + 1];
                    y[2 * i] = on0 ? fmaf(a, g.x, za * g.y) : a * g.x;
                    y[2 * i + 1] = on1 ? fmaf(b, g.z, zb * g.w) : b * g.z;
                }
                uint4 out;
                out.x = is_v ? raw[0] : pack_bf16x2(y[0], y[1]);
                out.y = is_v ? raw[1] : pack_bf16x2(y[2], y[3]);
                out.z = is_v ? raw[2] : pack_bf16x2(y[4], y[5]);
                out.w = is_v ? raw[3] : pack_bf16x2(y[6], y[7]);
                if (h >= end) continue;
                if (is_q) {
                    *reinterpret_cast<uint4 *>(p.q_out + (t * p.n_q_heads + h) * HD + d0) = out;
                    continue;
                }
                const int kvh = h - p.n_q_heads - (is_v ? p.n_kv_heads : 0);
                if (!is_v && p.k_out != nullptr)
                    *reinterpret_cast<uint4 *>(p.k_out + (t * p.n_kv_heads + kvh) * HD + d0) = out;
                if (!stored) continue;
                uint8_t *dst = (is_v ? p.v_cache : p.k_cache) + p.place.head_offset(slot, kvh);
                if (!p.fp8) {
                    *reinterpret_cast<uint4 *>(dst + d0 * 2) = out;
                } else {
                    const uint32_t o[4] = {out.x, out.y, out.z, out.w};
                    float e[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e[2 * i] = __uint_as_float(o[i] << 16);
                        e[2 * i + 1] = __uint_as_float(o[i] & 0xFFFF0000u);
                    }
                    if (!is_v && p.k_ref != nullptr) {
                        const float4 a = __ldg(reinterpret_cast<const float4 *>(p.k_ref + kvh * HD + d0));
                        const float4 b =
                            __ldg(reinterpret_cast<const float4 *>(p.k_ref + kvh * HD + d0 + 4));
                        const float ref[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) e[i] = __fsub_rn(e[i], ref[i]);
                    }
                    *reinterpret_cast<uint2 *>(dst + d0) =
                        make_uint2(f32x2_to_e4m3x2(e[0], e[1]) | (f32x2_to_e4m3x2(e[2], e[3]) << 16),
                                   f32x2_to_e4m3x2(e[4], e[5]) | (f32x2_to_e4m3x2(e[6], e[7]) << 16));
                }
            }
        }
    }
}

template <int HD>
cudaError_t launch(const Params &p, int mode, bool norm, unsigned grid, cudaStream_t stream) {
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, stream, p); };
    if (mode == kPairs)
        return norm ? go(rope_kernel<HD, kPairs, true>) : go(rope_kernel<HD, kPairs, false>);
    if (mode == kHalves)
        return norm ? go(rope_kernel<HD, kHalves, true>) : go(rope_kernel<HD, kHalves, false>);
    return norm ? go(rope_kernel<HD, kHalvesAny, true>) : go(rope_kernel<HD, kHalvesAny, false>);
}

}  // namespace rope

int launch_qk_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                   int64_t v_stride, const int32_t *positions, const int64_t *slot_mapping,
                   int64_t n, const attn_rope *r, const attn_kv_cache *cache, int n_q_heads,
                   int n_kv_heads, int head_dim, void *q_out, void *k_out, int32_t *err,
                   cudaStream_t stream) {
    rope::Params p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    p.positions = positions;
    p.inv_freq = r->inv_freq;
    p.q_weight = r->q_weight;
    p.k_weight = r->k_weight;
    p.factor = r->factor;
    p.eps = r->eps;
    p.rot = r->rot_dim;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.n_heads = n_q_heads + n_kv_heads;
    p.n = n;
    p.err = err;
    if (cache != nullptr) {
        p.n_heads += n_kv_heads;
        p.k_cache = static_cast<uint8_t *>(cache->k);
        p.v_cache = static_cast<uint8_t *>(cache->v);
        p.fp8 = cache->dtype == ATTN_KV_FP8_E4M3;
        p.k_ref = p.fp8 ? cache->k_ref : nullptr;
        p.slots = slot_mapping;
        p.num_slots = cache->num_slots;
        p.place = kv_place(cache, n_kv_heads, head_dim, p.fp8 ? 1 : 2);
    }
    const int mode = r->layout == ATTN_ROPE_PAIRS ? rope::kPairs
                     : r->rot_dim % 16 == 0       ? rope::kHalves
                                                  : rope::kHalvesAny;
    const int rows = 32 / (head_dim / 8), passes = (p.n_heads + rows - 1) / rows;
    // a token's passes are dealt to as many warps as the GPU holds at a time
    const int64_t blocks_held = (int64_t)device_sm_count() * rope::kBlocks;
    const int64_t chunks = std::min<int64_t>(
        passes, std::max<int64_t>(1, blocks_held * rope::kWarps / n));
    p.chunk_passes = (int)((passes + chunks - 1) / chunks);
    p.chunks = (passes + p.chunk_passes - 1) / p.chunk_passes;
    const int64_t blocks = (n * p.chunks + rope::kWarps - 1) / rope::kWarps;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, blocks_held);
    const bool norm = r->q_weight != nullptr || r->k_weight != nullptr;
    const cudaError_t e = head_dim == 128 ? rope::launch<128>(p, mode, norm, grid, stream)
                                          : rope::launch<64>(p, mode, norm, grid, stream);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace gqa
