// attend.cu -- decode attention fed from registers: 8-bit caches with a scale
// per block of tokens and head, and sliding windows with sinks.
//
// What is computed: for request b, query row r at position pos and query head
// h (KV head h / group),
//     out = sum_t softmax_t(scale * q . k_t) v_t   over the visible t:
//     t < seq_len, t <= pos, and t < n_sinks or window <= 0 or pos - t < window.
// With a scaled cache k_t = ks c_t, v_t = vs c'_t, the codes c being E4M3 or
// INT8 and ks, vs the scales of t's block.  Both scales leave the matrix
// products: scores are ks (q . c), and with x_t = scale ks (q . c) log2(e) and
// lv = log2(vs), the weights that meet the codes are
//     w_t = 2^(x_t + lv_t - M),  O = sum w_t c'_t,  l = sum w_t / vs_t,
// out = O / l.  M follows the maximum of x + lv, so w (rounded once to f16)
// stays in f16's range whatever the scales are, and l is a 32-bit sum.
//
// GB300 mapping.  A decode reads every key once and computes little with it:
// HBM bandwidth bounds it, so what counts is bytes in flight.  Each warp loads
// its keys straight from global memory into the registers of the mma.sync
// fragments that use them: the head dimension enters the k index of Q K^T in
// a permuted order (q's fragments in the same one) so that a thread's share of
// a key is whole 16-byte pieces, and every load instruction covers whole
// sectors.  No shared memory, barrier or copy engine stands between a load and
// its use: each warp runs alone over its own 16-key chunks, K of the next
// chunk requested as soon as Q K^T has consumed this one's, V after P V, and
// the 12 to 16 warps of an SM hide the latency of each other.  A row's address
// is its own, so pages of any size, rings and freed pages cost no other path.
//
// Work: a unit is (request, block of query rows, KV head).  All units' chunks
// are laid end to end and cut into equal shares, one per CTA of a persistent
// grid, whatever the lengths are; the four warps of a CTA take a share's
// chunks in turn and merge through shared memory.  A unit cut across CTAs
// leaves partial states that attend_merge_kernel adds in part order, so
// results do not depend on timing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace gqa {
namespace att {

constexpr int kChunk = 16;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxEntries = 256;  // (request, row block) pairs per launch
constexpr int kGapChunks = 8;     // what a change of unit costs a CTA, in chunks
constexpr int kMinChunks = 8;     // smallest share of a CTA
constexpr float kRescaleLog2 = 8.0f;  // the reference maximum moves past this only (w <= 2^8)
constexpr float kScaleFloor = 5.421010862427522e-20f;  // 2^-64, the smallest scale

enum Fmt { kBF16 = 0, kE4M3 = 1, kINT8 = 2 };

struct Params {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    const uint8_t *k, *v;
    const float *ks, *vs;  // [slot >> scale_shift][n_kv_heads], or nullptr (all 1)
    int scale_shift;
    int kind, slots_per_seq, block_size, max_blocks, num_pages;
    bool head_major;
    const int32_t *block_table, *seq_lens, *positions;
    int q_rows, n_q_heads, n_kv_heads, group, rows, row_blocks;
    int window, sinks, max_seq_len;
    int e0, n_entries;  // this launch's (request, row block) pairs
    int grid;
    float scale_log2;
    float *ws_o, *ws_lse;
    int2 *ws_parts;  // per unit: first and last CTA
    int32_t *err;
};

template <int FMT, int HD>
struct Geo {
    static constexpr int E = FMT == kBF16 ? 2 : 1;
    static constexpr int kRowBytes = HD * E;
    static constexpr int kKPieces = kRowBytes / 64;        // 16-byte pieces of a key per thread
    static constexpr int kStepsPerPiece = 4 / E;           // k-steps (of 16 dims) a piece feeds
    static constexpr int kVBytes = kRowBytes / 8 < 16 ? 8 : 16;  // a thread's V load
    static constexpr int kVPieces = kRowBytes / (8 * kVBytes);
    static constexpr int kVWords = kVBytes / 4;
    static constexpr int kVElems = kVBytes / E;            // dims of a V piece
};

// Bits 0 .. n - 1, n clamped to 0 .. 16.
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 16 ? 0xFFFFu : (1u << n) - 1u;
}

template <int BYTES>
__device__ __forceinline__ void load_piece(uint32_t *dst, const uint8_t *src, bool on) {
    if constexpr (BYTES == 16) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (on)
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                         : "l"(src));
        dst[0] = x.x, dst[1] = x.y, dst[2] = x.z, dst[3] = x.w;
    } else {
        uint2 x = make_uint2(0u, 0u);
        if (on)
            asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                         : "=r"(x.x), "=r"(x.y)
                         : "l"(src));
        dst[0] = x.x, dst[1] = x.y;
    }
}

// Four 8-bit codes -> two f16x2 words (bytes 0, 1 and bytes 2, 3); exact.
// INT8: a byte with its sign bit flipped is c + 128; behind the byte 0x64 it is
// the f16 1024 + (c + 128), from which 1152 is subtracted without rounding.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == kE4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(x));
    } else {
        x ^= 0x80808080u;
        const uint32_t bias = 0x64806480u;  // 1152, twice
        lo = __byte_perm(x, 0x64646464u, 0x4140u);
        hi = __byte_perm(x, 0x64646464u, 0x4342u);
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(bias));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(bias));
    }
}

// Whether a word of V holds a value that is not finite.
template <int FMT>
__device__ __forceinline__ bool word_not_finite(uint32_t w) {
    if constexpr (FMT == kBF16)
        return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
    else if constexpr (FMT == kE4M3)
        return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
    else
        return false;
}

template <int FMT>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
    if constexpr (FMT == kBF16)
        mma_bf16_16816(d, a, b0, b1);
    else
        mma_f16_16816(d, a, b0, b1);
}

// The visible keys of one (request, row block): [0, sinks) and [lo, hi), as
// chunks 0 .. sc - 1 and clo, clo + 1, ... (cnt chunks in all); pmin, pmax the
// rows' first and last position.
struct Entry {
    int cnt, sc, clo, lo, hi, pmin, pmax;
};

__device__ __forceinline__ Entry make_entry(const Params &p, int e, int rb_rows, bool report) {
    Entry t = {};
    const int b = e / p.row_blocks, rb = e - b * p.row_blocks;
    int len = p.seq_lens[b];
    const int cap = p.kind == ATTN_CACHE_LINEAR ? min(p.max_seq_len, p.slots_per_seq)
                                                : p.max_seq_len;
    if (len < 0 || len > cap) {
        if (report) report_error(p.err, ATTN_ERR_BOUNDS);
        len = max(0, min(len, cap));
    }
    const int row0 = rb * rb_rows, row1 = min(p.rows, row0 + rb_rows);
    t.pmin = INT32_MAX, t.pmax = -1;
    int oldest = INT32_MAX;  // of the rows that have a position
    for (int r = row0 / p.group; r <= (row1 - 1) / p.group; ++r) {
        const int pos = p.positions[(int64_t)b * p.q_rows + r];
        t.pmin = min(t.pmin, pos);
        t.pmax = max(t.pmax, pos);
        if (pos >= 0) oldest = min(oldest, pos);
    }
    t.hi = (int)min((int64_t)len, (int64_t)t.pmax + 1);
    if (t.hi <= 0) return t;
    t.lo = p.window > 0 ? max(0, min(t.hi, oldest - p.window + 1)) : 0;
    if (p.kind == ATTN_CACHE_RING)  // what the turning part of the ring still holds
        t.lo = max(t.lo, min(t.hi, len - (p.slots_per_seq - p.sinks)));
    const int chi = (t.hi + kChunk - 1) / kChunk;
    t.clo = t.lo / kChunk;
    t.sc = (min(p.sinks, t.hi) + kChunk - 1) / kChunk;
    if (t.clo <= t.sc) t.clo = t.sc = 0;  // one range: the keys between are masked
    if (t.sc == 0 && p.sinks <= 0) {
        t.cnt = t.lo < t.hi ? chi - t.clo : 0;
    } else {
        t.cnt = t.sc + (t.lo < t.hi || t.sc == 0 ? chi - t.clo : 0);
    }
    return t;
}

template <int FMT, int HD, int MT>
struct Smem {
    static constexpr int RB = MT == 0 ? 8 : 16;
    static constexpr int kStride = HD + 4;
    float o[kWarps][RB][kStride];
    float m[kWarps][RB], l[kWarps][RB], w[kWarps][RB], lse[RB];
    int prefix[kMaxEntries + 1];
    Entry entry[kMaxEntries];
};

template <int FMT, int HD, int MT>
__global__ void __launch_bounds__(kThreads, FMT == kBF16 ? (MT == 0 ? 3 : 2) : (MT == 0 ? 4 : 3))
    attend_kernel(const Params p) {
    using G = Geo<FMT, HD>;
    using S = Smem<FMT, HD, MT>;
    constexpr int RB = S::RB;
    constexpr int kSteps = HD / 16;
    __shared__ __align__(16) S sm;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;
    pdl_wait();
    pdl_launch_dependents();

    // ---- the launch's work, the same in every CTA
    for (int i = threadIdx.x; i < p.n_entries; i += kThreads)
        sm.entry[i] = make_entry(p, p.e0 + i, RB, blockIdx.x == 0);
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        if (lane == 0) sm.prefix[0] = 0;
        for (int base = 0; base < p.n_entries; base += 32) {
            const int i = base + lane;
            const int n = i < p.n_entries ? sm.entry[i].cnt : 0;
            int x = n > 0 ? (n + kGapChunks) * p.n_kv_heads : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (i < p.n_entries) sm.prefix[i + 1] = carry + x;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
    const int total = sm.prefix[p.n_entries];
    const int share = max(kMinChunks, (total + p.grid - 1) / p.grid);
    int g = min(total, (int)min((int64_t)blockIdx.x * share, (int64_t)total));
    const int g_end = min(total, g + share);

    if (blockIdx.x == 0) {
        // rows of a unit without keys are zeros, and it has no parts
        for (int i = warp; i < p.n_entries; i += kWarps) {
            if (sm.entry[i].cnt != 0) continue;
            const int e = p.e0 + i, b = e / p.row_blocks, rb = e - b * p.row_blocks;
            const int row0 = rb * RB, n = min(p.rows, row0 + RB) - row0;
            for (int kvh = 0; kvh < p.n_kv_heads; ++kvh) {
                if (lane == 0) p.ws_parts[i * p.n_kv_heads + kvh] = make_int2(0, -1);
                for (int j = lane; j < n * (HD / 8); j += 32) {
                    const int row = row0 + j / (HD / 8), r = row / p.group, gr = row - r * p.group;
                    reinterpret_cast<uint4 *>(
                        p.out + (((int64_t)b * p.q_rows + r) * p.n_q_heads + kvh * p.group + gr) *
                                    HD)[j % (HD / 8)] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    }

    while (g < g_end) {
        // ---- the next piece of a unit
        int lo_e = 0, hi_e = p.n_entries;
        while (hi_e - lo_e > 1) {
            const int mid = (lo_e + hi_e) >> 1;
            if (sm.prefix[mid] <= g) lo_e = mid; else hi_e = mid;
        }
        const Entry en = sm.entry[lo_e];
        const int span = en.cnt + kGapChunks;
        int off = g - sm.prefix[lo_e];
        const int kvh = off / span;
        off -= kvh * span;
        const int unit_start = g - off;
        if (off >= en.cnt) {  // in the gap behind the unit
            g = unit_start + span;
            continue;
        }
        const int c_end = min(en.cnt, off + (g_end - g));
        const int unit = lo_e * p.n_kv_heads + kvh;
        const int first = unit_start / share, last = (unit_start + en.cnt - 1) / share;
        const int e = p.e0 + lo_e, b = e / p.row_blocks, rb = e - b * p.row_blocks;
        const int row0 = rb * RB, n_rows = min(p.rows, row0 + RB) - row0;

        // ---- q fragments and positions
        const __nv_bfloat16 *qb =
            p.q + ((int64_t)b * p.q_rows * p.n_q_heads + kvh * p.group) * HD;
        auto row_of = [&](int rr) {  // row rr of the unit, in q and out
            const int row = row0 + min(rr, n_rows - 1), r = row / p.group;
            return ((int64_t)r * p.n_q_heads + (row - r * p.group)) * HD;
        };
        auto pos_of = [&](int rr) {
            return p.positions[(int64_t)b * p.q_rows + (row0 + min(rr, n_rows - 1)) / p.group];
        };
        constexpr int kQRows = MT == 0 ? 1 : 2;
        uint32_t qf[kSteps][2 * kQRows];
        bool q_big = false;
#pragma unroll
        for (int hr = 0; hr < kQRows; ++hr) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(qb + row_of(gq + 8 * hr));
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
                const int j = kk / G::kStepsPerPiece, s = kk % G::kStepsPerPiece;
                const int d0 = (16 / G::E) * (tq + 4 * j) + 4 * s;
                uint2 x = *reinterpret_cast<const uint2 *>(src + d0 / 2);
                if constexpr (FMT != kBF16) {  // f16 holds |q| < 65520
                    x.x = bf16x2_to_f16x2(x.x);
                    x.y = bf16x2_to_f16x2(x.y);
                    q_big |= (x.x & 0x7C00u) == 0x7C00u || (x.x & 0x7C000000u) == 0x7C000000u ||
                             (x.y & 0x7C00u) == 0x7C00u || (x.y & 0x7C000000u) == 0x7C000000u;
                }
                qf[kk][hr] = x.x;
                qf[kk][kQRows + hr] = x.y;
            }
        }
        if (q_big) report_error(p.err, ATTN_ERR_UNSUPPORTED);
        int rpos[2];  // positions of the two rows this thread keeps scores of
        rpos[0] = MT == 0 ? pos_of(2 * tq) : pos_of(gq);
        rpos[1] = MT == 0 ? pos_of(2 * tq + 1) : pos_of(gq + 8);

        // ---- where chunks lie
        const int32_t *bt = p.block_table + (int64_t)b * p.max_blocks;
        const int blk_rows = p.kind == ATTN_CACHE_PAGED ? p.block_size : p.slots_per_seq;
        const uint32_t row_step = p.head_major ? 1u : (uint32_t)p.n_kv_heads;
        // a chunk's 16 rows are evenly spaced
        const bool even = p.kind == ATTN_CACHE_LINEAR ||
                          (p.kind == ATTN_CACHE_PAGED && p.block_size % kChunk == 0);
        auto row_index = [&](int block, int r) -> uint32_t {  // in rows of one head
            return p.head_major ? ((uint32_t)block * p.n_kv_heads + kvh) * blk_rows + r
                                : ((uint32_t)block * blk_rows + r) * p.n_kv_heads + kvh;
        };
        auto chunk_t0 = [&](int c) { return (c < en.sc ? c : c - en.sc + en.clo) * kChunk; };
        auto chunk_mask = [&](int t0) -> uint32_t {
            return (bits_below(p.sinks - t0) | (0xFFFFu & ~bits_below(en.lo - t0))) &
                   bits_below(en.hi - t0);
        };
        // the table entry of an evenly spaced chunk (read a chunk ahead of its rows)
        auto chunk_page = [&](int c) -> int {
            if (p.kind != ATTN_CACHE_PAGED || !even || c >= c_end) return b;
            return __ldg(bt + chunk_t0(c) / p.block_size);
        };

        float o[MT == 0 ? HD / 16 : HD / 8][4];
#pragma unroll
        for (auto &x : o) x[0] = x[1] = x[2] = x[3] = 0.f;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

        // the chunk in flight
        uint32_t kw[2][4 * G::kKPieces], vw[4][G::kVWords * G::kVPieces];
        uint32_t mask = 0, base = 0, spread = 0;
        float sk = 1.f, sv = 1.f;
        int t0 = 0;
        // finds chunk c's rows: even chunks have row `base + key * row_step`,
        // others lane key & 15 holds row `spread`; `mask` the keys present
        auto locate = [&](int c, int page) {
            t0 = chunk_t0(c);
            mask = chunk_mask(t0);
            int slot = 0;
            if (even) {
                if (p.kind == ATTN_CACHE_PAGED) {
                    if ((unsigned)page >= (unsigned)p.num_pages) {
                        if (lane == 0) report_error(p.err, ATTN_ERR_BOUNDS);
                        mask = 0, page = 0;
                    }
                    const int r = t0 % p.block_size;
                    base = row_index(page, r);
                    slot = page * p.block_size + r;
                } else {
                    base = row_index(b, t0);
                    slot = b * p.slots_per_seq + t0;
                }
            } else {
                const int t = t0 + (lane & 15);
                bool on = (mask >> (lane & 15)) & 1u;
                spread = 0;
                if (on) {
                    if (p.kind == ATTN_CACHE_PAGED) {
                        const int pi = t / p.block_size, id = __ldg(bt + pi);
                        if ((unsigned)id >= (unsigned)p.num_pages) {
                            report_error(p.err, ATTN_ERR_BOUNDS);
                            on = false;
                        } else {
                            spread = row_index(id, t - pi * p.block_size);
                        }
                    } else {
                        spread = row_index(b, t < p.sinks ? t
                                                          : p.sinks + (t - p.sinks) %
                                                                          (p.slots_per_seq - p.sinks));
                    }
                }
                mask = __ballot_sync(0xffffffffu, on) & 0xFFFFu;
            }
            if constexpr (FMT != kBF16) {
                if (p.ks != nullptr && mask != 0) {
                    const int64_t i = (int64_t)(slot >> p.scale_shift) * p.n_kv_heads + kvh;
                    sk = __ldg(p.ks + i);
                    sv = __ldg(p.vs + i);
                }
            }
        };
        auto row_ptr = [&](const uint8_t *cache, int key) {
            const uint32_t r = even ? base + key * row_step : __shfl_sync(0xffffffffu, spread, key);
            return cache + (uint64_t)r * G::kRowBytes;
        };
        auto load_k = [&]() {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = gq + 8 * h;
                const uint8_t *src = row_ptr(p.k, key) + tq * 16;
                const bool on = (mask >> key) & 1u;
#pragma unroll
                for (int j = 0; j < G::kKPieces; ++j)
                    load_piece<16>(&kw[h][4 * j], src + 64 * j, on);
            }
        };
        auto load_v = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 2 * tq + (i & 1) + 8 * (i >> 1);
                const uint8_t *src = row_ptr(p.v, key) + gq * G::kVBytes;
                const bool on = (mask >> key) & 1u;
#pragma unroll
                for (int j = 0; j < G::kVPieces; ++j)
                    load_piece<G::kVBytes>(&vw[i][G::kVWords * j], src + 8 * G::kVBytes * j, on);
            }
        };

        const int c0 = off + warp;
        int page = chunk_page(c0);
        if (c0 < c_end) {
            locate(c0, page);
            load_k();
            load_v();
        }
        page = chunk_page(c0 + kWarps);
        for (int c = c0; c < c_end; c += kWarps) {
            const bool more = c + kWarps < c_end;
            const uint32_t cur_mask = mask;
            const int cur_t0 = t0;
            const float cur_sk = sk, cur_sv = fmaxf(sv, kScaleFloor);
            // ---- scores: MT 0 keys are the rows of S^T = K Q^T, MT 1 the columns of S = Q K^T
            float s[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
                const int j = kk / G::kStepsPerPiece, st = kk % G::kStepsPerPiece;
                uint32_t x[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (FMT == kBF16) {
                        x[h][0] = kw[h][4 * j + 2 * st];
                        x[h][1] = kw[h][4 * j + 2 * st + 1];
                    } else {
                        codes_to_f16<FMT>(kw[h][4 * j + st], x[h][0], x[h][1]);
                    }
                }
                if constexpr (MT == 0) {
                    const uint32_t a[4] = {x[0][0], x[1][0], x[0][1], x[1][1]};
                    mma16<FMT>(s[kk & 1], a, qf[kk][0], qf[kk][1]);
                } else {
                    mma16<FMT>(s[0], qf[kk], x[0][0], x[0][1]);
                    mma16<FMT>(s[1], qf[kk], x[1][0], x[1][1]);
                }
            }
            if constexpr (MT == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[0][i] += s[1][i];
            }
            // ---- the next chunk's keys
            if (more) {
                locate(c + kWarps, page);
                load_k();
            }
            page = chunk_page(c + 2 * kWarps);
            // ---- mask and weights.  x(row, key): element (i, j) of the thread is
            // MT 0: row i & 1, key gq + 8 (i >> 1); MT 1: row i >> 1, key 8 j + 2 tq + (i & 1)
            constexpr int NJ = MT == 0 ? 1 : 2;
            const float f = cur_sk * p.scale_log2;
            float lv = 0.f, inv_sv = 1.f;
            if constexpr (FMT != kBF16) {
                lv = __log2f(cur_sv);
                inv_sv = __frcp_rn(cur_sv);
            }
            const bool open = cur_mask == 0xFFFFu && cur_t0 + kChunk - 1 <= en.pmin &&
                              (p.window <= 0 || en.pmax - cur_t0 < p.window ||
                               cur_t0 + kChunk <= p.sinks);
            auto row_i = [](int i) { return MT == 0 ? (i & 1) : (i >> 1); };
            auto sees = [&](int i_row, int key) {
                const int t = cur_t0 + key, pos = rpos[i_row];
                return ((cur_mask >> key) & 1u) && t <= pos &&
                       (p.window <= 0 || pos - t < p.window || t < p.sinks);
            };
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j][i] = fmaf(s[j][i], f, lv);
            if (!open) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = MT == 0 ? gq + 8 * (i >> 1) : 8 * j + 2 * tq + (i & 1);
                        s[j][i] = sees(row_i(i), key) ? s[j][i] : -INFINITY;
                    }
            }
            float alpha[2];
            bool moved = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx;
                if constexpr (MT == 0) {
                    mx = fmaxf(s[0][r], s[0][r + 2]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                } else {
                    mx = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]),
                               fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                }
                const float m_old = m_run[r];
                const float m_new = mx > m_old + kRescaleLog2 ? mx : m_old;
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                alpha[r] = m_new == m_old ? 1.f : fast_exp2(m_old - m_use);
                moved |= m_new != m_old;
                m_run[r] = m_new;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (row_i(i) == r) {
                            s[j][i] = fast_exp2(s[j][i] - m_use);
                            sum += s[j][i];
                        }
                l_run[r] = l_run[r] * alpha[r] + sum * inv_sv;
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (auto &x : o)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] *= alpha[row_i(i)];
            }
            // ---- weights as the operand of P V: f16 (one rounding: 11 bits), or for
            // a bf16 cache two bf16 halves (16 bits), since one bf16 rounding of P
            // would cost as much as the output's own
            constexpr int NP = MT == 0 ? 2 : 4;
            uint32_t ph[NP], pl[NP];
            if constexpr (MT == 0) {
                if constexpr (FMT == kBF16) {
                    split_bf16x2(s[0][0], s[0][1], ph[0], pl[0]);
                    split_bf16x2(s[0][2], s[0][3], ph[1], pl[1]);
                    pl[0] = movmatrix_trans(pl[0]);
                    pl[1] = movmatrix_trans(pl[1]);
                } else {
                    ph[0] = pack_f16x2(s[0][0], s[0][1]);
                    ph[1] = pack_f16x2(s[0][2], s[0][3]);
                }
                ph[0] = movmatrix_trans(ph[0]);
                ph[1] = movmatrix_trans(ph[1]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = i >> 1, r = i & 1;
                    if constexpr (FMT == kBF16)
                        split_bf16x2(s[j][2 * r], s[j][2 * r + 1], ph[i], pl[i]);
                    else
                        ph[i] = pack_f16x2(s[j][2 * r], s[j][2 * r + 1]);
                }
            }
            // V operands of two neighbouring dims (word w of the pieces): x[0] and
            // x[1] dim 0 and 1 over keys 2 tq, 2 tq + 1, x[2] and x[3] over + 8
            auto v_pair = [&](const uint32_t (&w)[4], int hi, uint32_t (&x)[4]) {
                if constexpr (FMT == kBF16) {
                    x[0] = __byte_perm(w[0], w[1], 0x5410u);
                    x[1] = __byte_perm(w[0], w[1], 0x7632u);
                    x[2] = __byte_perm(w[2], w[3], 0x5410u);
                    x[3] = __byte_perm(w[2], w[3], 0x7632u);
                } else {
                    const uint32_t sel = hi ? 0x7362u : 0x5140u;
                    codes_to_f16<FMT>(__byte_perm(w[0], w[1], sel), x[0], x[1]);
                    codes_to_f16<FMT>(__byte_perm(w[2], w[3], sel), x[2], x[3]);
                }
            };
            constexpr int kPairs = HD / 16;            // pairs of dims of a thread
            constexpr int kPairsPerWord = 2 / G::E;
            auto add_pv = [&](int d, const uint32_t (&x)[4], float (&oa)[4], float (&ob)[4]) {
                if constexpr (MT == 0) {  // rows of O^T: dim 0 in elements 0, 1, dim 1 in 2, 3
                    mma16<FMT>(oa, x, ph[0], ph[1]);
                    if constexpr (FMT == kBF16) mma16<FMT>(oa, x, pl[0], pl[1]);
                } else {
                    mma16<FMT>(oa, ph, x[0], x[2]);
                    mma16<FMT>(ob, ph, x[1], x[3]);
                    if constexpr (FMT == kBF16) {
                        mma16<FMT>(oa, pl, x[0], x[2]);
                        mma16<FMT>(ob, pl, x[1], x[3]);
                    }
                }
            };
            if constexpr (FMT != kINT8) {
                if (!open) {
                    // A value that is not finite reaches only the rows that see its
                    // key: 0 times it would be NaN in every row.  Such keys are
                    // multiplied alone, added where seen, and taken out.
                    uint32_t odd = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int w = 0; w < G::kVWords * G::kVPieces; ++w)
                            if (word_not_finite<FMT>(vw[i][w]))
                                odd |= 1u << (2 * tq + (i & 1) + 8 * (i >> 1));
                    odd = __reduce_or_sync(0xffffffffu, odd);
                    while (odd != 0) {
                        const int n = __ffs(odd) - 1;
                        odd &= odd - 1;
#pragma unroll
                        for (int d = 0; d < kPairs; ++d) {
                            uint32_t w[4], x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                w[i] = n == 2 * tq + (i & 1) + 8 * (i >> 1)
                                           ? vw[i][d / kPairsPerWord]
                                           : 0u;
                            v_pair(w, d % kPairsPerWord, x);
                            float ta[4] = {0.f, 0.f, 0.f, 0.f}, tb[4] = {0.f, 0.f, 0.f, 0.f};
                            add_pv(d, x, ta, tb);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (sees(row_i(i), n)) {
                                    o[MT == 0 ? d : 2 * d][i] += ta[i];
                                    if constexpr (MT != 0) o[2 * d + 1][i] += tb[i];
                                }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (n == 2 * tq + (i & 1) + 8 * (i >> 1))
#pragma unroll
                                for (int w = 0; w < G::kVWords * G::kVPieces; ++w) vw[i][w] = 0u;
                    }
                }
            }
#pragma unroll
            for (int d = 0; d < kPairs; ++d) {
                uint32_t w[4], x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = vw[i][d / kPairsPerWord];
                v_pair(w, d % kPairsPerWord, x);
                if constexpr (MT == 0)
                    add_pv(d, x, o[d], o[d]);
                else
                    add_pv(d, x, o[2 * d], o[2 * d + 1]);
            }
            if (more) load_v();
        }

        // ---- the four warps' states -> one
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if constexpr (MT == 0) {
                l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 4);
                l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 8);
                l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 16);
            } else {
                l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 1);
                l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 2);
            }
            const int row = MT == 0 ? 2 * tq + r : gq + 8 * r;
            if (MT == 0 ? gq == 0 : tq == 0) {
                sm.m[warp][row] = m_run[r];
                sm.l[warp][row] = l_run[r];
            }
        }
        // dim of element e of V piece j of thread group g8
        auto dim_of = [](int g8, int d) {  // d: dim index 0 .. HD / 8 - 1 of the group
            return G::kVElems * (g8 + 8 * (d / G::kVElems)) + d % G::kVElems;
        };
        if constexpr (MT == 0) {
#pragma unroll
            for (int d = 0; d < HD / 16; ++d)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    *reinterpret_cast<float2 *>(&sm.o[warp][2 * tq + r][dim_of(gq, 2 * d)]) =
                        make_float2(o[d][r], o[d][r + 2]);
        } else {
#pragma unroll
            for (int d = 0; d < HD / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float2 *>(
                        &sm.o[warp][gq + 8 * (i >> 1)][dim_of(2 * tq + (i & 1), 2 * d)]) =
                        make_float2(o[2 * d][i], o[2 * d + 1][i]);
        }
        __syncthreads();
        if (threadIdx.x < RB) {
            const int row = threadIdx.x;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][row]);
            const float m_use = m == -INFINITY ? 0.f : m;
            float f[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                f[w] = fast_exp2(sm.m[w][row] - m_use);
                l += f[w] * sm.l[w][row];
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sm.w[w][row] = f[w] * inv;
            sm.lse[row] = l == 0.f ? -INFINITY : m_use + log2f(l);
        }
        __syncthreads();
        const bool whole = first == last;
        const int64_t slot = unit + blockIdx.x;  // unique: shares are contiguous
        for (int i = threadIdx.x; i < n_rows * (HD / 4); i += kThreads) {
            const int row = i / (HD / 4), d = (i % (HD / 4)) * 4;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 x = *reinterpret_cast<const float4 *>(&sm.o[w][row][d]);
                const float f = sm.w[w][row];
                a.x += f * x.x, a.y += f * x.y, a.z += f * x.z, a.w += f * x.w;
            }
            if (whole) {
                uint2 y;
                y.x = pack_bf16x2(a.x, a.y);
                y.y = pack_bf16x2(a.z, a.w);
                *reinterpret_cast<uint2 *>(
                    p.out + ((int64_t)b * p.q_rows * p.n_q_heads + kvh * p.group) * HD +
                    row_of(row) + d) = y;
            } else {
                *reinterpret_cast<float4 *>(p.ws_o + (slot * RB + row) * HD + d) = a;
            }
        }
        if (!whole && threadIdx.x < n_rows) p.ws_lse[slot * RB + threadIdx.x] = sm.lse[threadIdx.x];
        if (off == 0 && threadIdx.x == 0) p.ws_parts[unit] = make_int2(first, last);
        __syncthreads();  // the shared states are free again
        g += c_end - off;
    }
}

// Adds the partial states of every unit that more than one CTA held: a warp
// per (unit, row), its lanes along the head, parts in CTA order.
template <int HD, int RB>
__global__ void __launch_bounds__(256) attend_merge_kernel(const Params p) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int V = HD / 32;  // dims of a lane
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t unit = i / RB;
    const int row = (int)(i - unit * RB);
    if (unit >= (int64_t)p.n_entries * p.n_kv_heads) return;
    const int2 parts = p.ws_parts[unit];
    if (parts.y <= parts.x) return;
    const int entry = (int)(unit / p.n_kv_heads), kvh = (int)(unit - (int64_t)entry * p.n_kv_heads);
    const int e = p.e0 + entry, b = e / p.row_blocks, rb = e - b * p.row_blocks;
    const int q_row = rb * RB + row;
    if (q_row >= p.rows) return;
    float m = -INFINITY;
    for (int c = parts.x + lane; c <= parts.y; c += 32)
        m = fmaxf(m, __ldcg(p.ws_lse + (unit + c) * RB + row));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.f;  // no part has a key: every weight below is 0
    float acc[V] = {}, sum = 0.f;
#pragma unroll 8
    for (int c = parts.x; c <= parts.y; ++c) {
        const int64_t at = (unit + c) * RB + row;
        const float f = fast_exp2(__ldcg(p.ws_lse + at) - m);
        sum += f;
        const float *src = p.ws_o + at * HD + lane * V;
        if constexpr (V == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
            acc[0] += f * x.x, acc[1] += f * x.y, acc[2] += f * x.z, acc[3] += f * x.w;
        } else {
            const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
            acc[0] += f * x.x, acc[1] += f * x.y;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int r = q_row / p.group;
    uint32_t *dst = reinterpret_cast<uint32_t *>(
        p.out + (((int64_t)b * p.q_rows + r) * p.n_q_heads + kvh * p.group + (q_row - r * p.group)) *
                    HD + lane * V);
#pragma unroll
    for (int d = 0; d < V / 2; ++d) dst[d] = pack_bf16x2(acc[2 * d] * inv, acc[2 * d + 1] * inv);
}

template <int FMT, int HD, int MT>
int launch(const Params &p, bool merge, cudaStream_t stream) {
    constexpr int RB = MT == 0 ? 8 : 16;
    if (launch_pdl(attend_kernel<FMT, HD, MT>, dim3((unsigned)p.grid), dim3(kThreads), 0, stream,
                   p) != cudaSuccess)
        return ATTN_ERR_CUDA;
    if (!merge) return ATTN_OK;
    const int64_t warps = (int64_t)p.n_entries * p.n_kv_heads * RB;
    return launch_pdl(attend_merge_kernel<HD, RB>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0,
                      stream, p) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

}  // namespace att

int plan_attend(const attn_kv_cache *cache, int batch, int q_rows, int n_q_heads, int n_kv_heads,
                int head_dim, int max_seq_len, int window, int sinks, AttendPlan *plan) {
    const int64_t rows = (int64_t)q_rows * (n_q_heads / n_kv_heads);
    plan->mt = rows <= 8 ? 0 : 1;
    const int rb = plan->mt == 0 ? 8 : 16;
    const int64_t row_blocks = (rows + rb - 1) / rb;
    // the most chunks an entry can have, and the most it has when its rows are neighbours
    const int64_t chunks = ((int64_t)max_seq_len + att::kChunk - 1) / att::kChunk + 1;
    int64_t usual = chunks;
    if (window > 0)
        usual = std::min<int64_t>(chunks, ((int64_t)window + q_rows + sinks) / att::kChunk + 3);
    const int64_t entries = (int64_t)batch * row_blocks;
    // rows of one head and prefixes of chunks are counted in 32 bits
    const int64_t per_entry = (chunks + att::kGapChunks) * n_kv_heads;
    if (rows >= (int64_t(1) << 31) || entries >= (int64_t(1) << 31) ||
        per_entry >= (int64_t(1) << 30) ||
        cache->num_slots * n_kv_heads >= (int64_t(1) << 32))
        return ATTN_ERR_SHAPE;
    plan->row_blocks = (int)row_blocks;
    plan->entries = (int)entries;
    plan->per_launch = (int)std::max<int64_t>(
        1, std::min<int64_t>(std::min<int64_t>(entries, att::kMaxEntries),
                             (int64_t(1) << 30) / per_entry));
    const bool bf16 = cache->dtype == ATTN_KV_BF16;
    const int per_sm = bf16 ? (plan->mt == 0 ? 3 : 2) : (plan->mt == 0 ? 4 : 3);
    const int64_t needed = ((int64_t)plan->per_launch * (usual + att::kGapChunks) * n_kv_heads +
                            att::kMinChunks - 1) / att::kMinChunks;
    plan->grid = (int)std::max<int64_t>(
        1, std::min<int64_t>(needed, (int64_t)per_sm * device_sm_count()));
    plan->merge = plan->grid > 1;
    const size_t units = (size_t)plan->per_launch * n_kv_heads, slots = units + plan->grid;
    // behind the counters of attn_decode's other kernels, which have to stay zero
    // in a workspace that serves both
    DecodePlan dp;
    plan_decode(cache, batch, q_rows, n_q_heads, n_kv_heads, head_dim, max_seq_len, window, &dp);
    plan->parts_offset = (dp.counter_bytes + 255) & ~size_t(255);
    plan->lse_offset = (plan->parts_offset + units * sizeof(int2) + 255) & ~size_t(255);
    plan->o_offset = (plan->lse_offset + slots * rb * sizeof(float) + 255) & ~size_t(255);
    plan->workspace = plan->o_offset + slots * rb * (size_t)head_dim * sizeof(float);
    plan->launches = (plan->entries + plan->per_launch - 1) / plan->per_launch * (plan->merge ? 2 : 1);
    return ATTN_OK;
}

int launch_attend(const AttendPlan &plan, const void *q, const attn_kv_cache *cache,
                  const int32_t *seq_lens, const int32_t *positions, int q_rows, int max_seq_len,
                  int window, int sinks, int n_q_heads, int n_kv_heads, int head_dim, float scale,
                  void *out, void *workspace, int32_t *err, cudaStream_t stream) {
    att::Params p = {};
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
    p.head_major = cache->layout == ATTN_LAYOUT_BHSD;
    p.block_table = cache->kind == ATTN_CACHE_PAGED ? cache->block_table : nullptr;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.q_rows = q_rows;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = n_q_heads / n_kv_heads;
    p.rows = q_rows * p.group;
    p.row_blocks = plan.row_blocks;
    p.window = window;
    p.sinks = window > 0 ? sinks : 0;  // without a window every key is visible
    p.max_seq_len = max_seq_len;
    p.grid = plan.grid;
    p.scale_log2 = scale * 1.4426950408889634f;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.ws_parts = reinterpret_cast<int2 *>(ws + plan.parts_offset);
    p.ws_lse = reinterpret_cast<float *>(ws + plan.lse_offset);
    p.ws_o = reinterpret_cast<float *>(ws + plan.o_offset);
    p.err = err;
    const int fmt = cache->dtype == ATTN_KV_BF16          ? att::kBF16
                    : cache->dtype == ATTN_KV_INT8_SCALED ? att::kINT8
                                                          : att::kE4M3;
    for (p.e0 = 0; p.e0 < plan.entries; p.e0 += plan.per_launch) {
        p.n_entries = std::min(plan.per_launch, plan.entries - p.e0);
        int rc = ATTN_ERR_UNSUPPORTED;
        auto run = [&](auto fmt_c) {
            constexpr int F = decltype(fmt_c)::value;
            if (head_dim == 128)
                rc = plan.mt == 0 ? att::launch<F, 128, 0>(p, plan.merge, stream)
                                  : att::launch<F, 128, 1>(p, plan.merge, stream);
            else
                rc = plan.mt == 0 ? att::launch<F, 64, 0>(p, plan.merge, stream)
                                  : att::launch<F, 64, 1>(p, plan.merge, stream);
        };
        if (fmt == att::kBF16)
            run(std::integral_constant<int, att::kBF16>{});
        else if (fmt == att::kE4M3)
            run(std::integral_constant<int, att::kE4M3>{});
        else
            run(std::integral_constant<int, att::kINT8>{});
        if (rc != ATTN_OK) return rc;
    }
    return ATTN_OK;
}

}  // namespace gqa
