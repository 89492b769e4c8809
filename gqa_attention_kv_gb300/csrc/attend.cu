// attend.cu -- decode attention over 8-bit caches with a scale per block of tokens
// and head, and under sliding windows with sinks.
//
// What is computed: for request b, query row r at position pos and query head
// h (KV head h / group),
//     out = sum_t softmax_t(scale * q . k_t) v_t   over the visible t:
//     t < seq_len, t <= pos, and t < n_sinks or window <= 0 or pos - t < window.
// With a scaled cache k_t = ks c_t, v_t = vs c'_t, the codes c being E4M3 or
// INT8 and ks, vs the scales of t's block.  Both scales leave the matrix
// products: scores are ks (q . c), and with x_t = scale ks (q . c) log2(e) and
// lv = log2(vs), the weights that meet the codes are (but for a constant factor)
//     w_t = 2^(x_t + lv_t - M),  O = sum w_t c'_t,  l = sum w_t / vs_t,
// out = O / l.  M follows the maximum of x + lv, so w (rounded once to f16)
// stays in f16's range whatever the scales are, and l is a 32-bit sum.
//
// GB300 mapping.  A decode reads every key once and computes little with it: HBM
// bandwidth is its floor, and what stands before the floor is the work of a
// warp per key (unpacking codes, mma.sync fragments, the softmax), so the kernel
// is built for many bytes in flight and few instructions a key:
//   * Each warp runs alone over its own chunks of 16 keys and copies them into
//     its own ring in shared memory with cp.async, 4 KB of K and 4 KB of V a step
//     for 8-bit caches (32 keys of 128 dims), one step ahead (two for bf16).  No
//     barrier stands between a copy and its use, a row's address is its own (pages
//     of any size, rings and freed pages need no other kernel), and a step whose
//     keys are all there and evenly spaced takes a path without per-key checks.
//   * The head dimension enters the k index of Q K^T in a permuted order (q's
//     fragments in the same one), so a thread's share of a key is whole 16-byte
//     pieces: one LDS.128 feeds four k-steps, and codes become f16 fragments in
//     registers, two instructions a four codes (E4M3) or three to five (INT8).
//     V's codes of two keys are interleaved bytewise before they are converted,
//     so no transposing load is needed.
//   * Up to 8 query rows (MT 0) keys are the rows of the products, S^T = K Q^T
//     and O^T = V^T P^T; up to 16 (MT 1) the query rows are.
//   * A score's softmax reference moves only past 2^8 (lazily), and a step that
//     every row sees whole is not masked.
//   * What is the same for all of a chunk's keys (its first row through the table,
//     whether they are all visible, its scales with their logarithm and inverse) is
//     worked out by one lane for each of the next 32 chunks, and shuffled.
// Measured against earlier forms of this kernel (64 requests x 4 rows, 64 to 4,096
// INT8 keys, 8 KV heads of 128, pages of 16; floor 41 us): keys loaded into the
// fragments' registers one step ahead 127 us, in the ring 82, with in-kernel merging
// and steps without per-key checks 74, with 32 keys a step on twelve warps an SM
// instead of 16 on sixteen 63, with a lane for each of 32 chunks' rows and scales (13%
// fewer instructions a key; 20% at head_dim 64) 60, with the shares cut anew 58 to 59 (4.7
// TB/s).  One query row: 5.2 TB/s E4M3, 5.9 bf16 (64 x 2,080 keys).  What bounds it
// now: the warps' own dependency chains (issue slots about half used), and at one row
// a KV head DRAM.
//
// Work: a unit is (request, block of query rows, one or two KV heads).  All units'
// chunks are laid end to end and cut into equal shares, one per CTA of a
// persistent grid, whatever the lengths are; the four warps of a CTA take a
// share's chunks in turn (two warps a head where a unit has two) and merge
// through shared memory.  A unit cut across CTAs leaves partial states that the
// CTA storing the last of them adds up, in part order, so results do not depend
// on timing; units that may lie in very many parts are left to
// attend_merge_kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace gqa {
namespace att {

constexpr int kChunk = 16;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxEntries = 128;  // (request, row block) pairs per launch
constexpr int kPartEntries = 256;  // ... of launch_attend_parts (its shared memory allows that)
// What a change of unit costs a CTA, in chunks: in the share arithmetic every unit is
// followed by so many of nothing.  64 ragged requests (64 to 4,096 keys): 65.1 us with
// 16, 60.3 with 24, 59.0 with 28, 58.3 with 32, 59.4 with 36; 64 even ones (2,080 keys)
// 57.6 with 24, 57.1 with 32.
constexpr int kGapChunks = 32;
// Smallest share of a CTA, with 2, 4 and 8 chunks: one request of 9,000 tokens under a
// window of 1,024 9.05, 9.06 and 8.6 us; 512 E4M3 keys 8.4, 7.2 and 7.0; four requests of
// 300 8.7, 8.75 and 8.4; two of 700 with 64 dims in bf16 11.1, 9.9 and 10.1.
constexpr int kMinChunks = 4;
// Parts of a unit that its last CTA adds up itself.  17 parts: 8.9 us of GPU time
// against 8.3 with the merge kernel, which costs the host 3 us to launch; 76 parts:
// 22.5 against 16.4 us.  The host decides by the longest that units can be; where one is
// much longer than the others are, shares are cut so that it has no more parts (40
// requests, one of 20,000 keys among 5 to 19: 21.5 us, 46 with shares of the sum alone).
constexpr int kKernelParts = 24;
constexpr float kRescaleLog2 = 8.0f;  // the reference maximum moves past this only (w <= 2^8)
// f16 weights are held times 2^7, 2^15 at most: those above 2^-21 of the largest keep
// f16's 11 bits (2^-14 without), however small the largest's own value is
constexpr float kWeightLog2 = 7.0f;
// Scores (times log2(e)) up to which a weight is right: it is exp2 of the exact s f - M, and
// half a step of M has to leave it below 2^16 (f16) or 2^128.  Larger ones are reported, also
// where a K scale is so large that its factor f is cut off for s f to stay finite.
constexpr float kScoreTopF16 = 0x1p24f, kScoreTopBf16 = 0x1p30f;
constexpr float kFactorTop = 0x1p90f;
constexpr float kPartWeight = 0x1p-12f;  // of the largest part: the sum of 4,096 outputs is finite
// Weights of outputs that are added up are no smaller: 0 times an infinite one would be NaN
constexpr float kSmallest = 0x1p-149f;
constexpr float kScaleFloor = 5.421010862427522e-20f;  // 2^-64, the smallest scale

enum Fmt { kBF16 = 0, kE4M3 = 1, kINT8 = 2 };

struct Params {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    const uint8_t *k, *v;
    const float *ks, *vs;  // [slot >> scale_shift][n_kv_heads], or nullptr (all 1)
    int scale_shift;
    int kind, slots_per_seq, block_size, max_blocks, num_pages;
    // pages of whole chunks: n / page_chunks = umulhi(n << 4, page_mul) >> page_shift, n < 2^28
    int page_chunks, page_shift;
    uint32_t page_mul;
    bool head_major;
    const int32_t *block_table, *seq_lens, *positions;
    int q_rows, n_q_heads, n_kv_heads, group, rows, row_blocks;
    int n_groups;  // KV heads by the heads of a unit
    int window, sinks, max_seq_len;
    int e0, n_entries;  // this launch's (request, row block) pairs
    int grid;
    float scale_log2;
    float *ws_o, *ws_lse;
    int2 *ws_parts;     // per unit: first and last CTA (merge kernel)
    int32_t *ws_count;  // per unit: parts stored (0 between calls), or nullptr: merge kernel
    // only keys t >= from[b] (clipped to 0 .. from_cap), every unit left as parts; or nullptr
    const int32_t *from;
    int from_cap;
    // (kParts) This launch reads and writes nothing that the one before it writes, and that one let
    // it begin behind its own wait for everything earlier: it is waited for last, so that whoever
    // waits for this launch has waited for both
    bool late_wait;
    // (kParts) shares, `pieces` of them, are taken one after another by whichever
    // CTA is free (`next` counts them, from the 0 at which the merge of the call before left it),
    // so CTAs that start late do no harm; else one each
    int32_t *next;
    int pieces;
    int32_t *err;
};

// A stage of a warp's ring: the K rows and the V rows of a step, NSUB chunks.  Thread
// (gq, tq) reads pieces tq + 4 j of K rows gq and gq + 8, and piece gq (+ 8 j)
// of V rows 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9; rows are swizzled so that the
// lanes of one access meet different banks.
template <int FMT, int HD, int MT, int HG>
struct Geo {
    static constexpr int E = FMT == kBF16 ? 2 : 1;
    static constexpr int RB = MT == 0 ? 8 : 16;                  // query rows of a unit
    static constexpr int kRowBytes = HD * E;
    static constexpr int kKPieces = kRowBytes / 64;              // 16-byte pieces of a key a thread
    static constexpr int kStepsPerPiece = 4 / E;                 // k-steps (of 16 dims) of a piece
    static constexpr int kVBytes = kRowBytes / 8 < 16 ? 8 : 16;  // a V piece
    static constexpr int kVPieces = kRowBytes / (8 * kVBytes);
    static constexpr int kVWords = kVBytes / 4 * kVPieces;       // words of a key a thread
    static constexpr int kVElems = kVBytes / E;                  // dims of a V piece
    // chunks of a step: 4 KB of K, but for bf16 rows of 128 bytes
    static constexpr int NSUB = kRowBytes == 64 ? 4 : FMT != kBF16 ? 2 : 1;
    static constexpr int kChunkBytes = kChunk * kRowBytes;
    static constexpr int kStepBytes = NSUB * kChunkBytes;        // K (or V) of a step
    // Stages and blocks an SM share its 227 KB: 8-bit steps take long enough that twelve
    // warps one step ahead do better than eight two steps ahead (64 ragged requests x 4
    // rows 59.4 us, 64.5; 32 heads of 64 65.0, 67.2), bf16 steps do not (64 x 8 heads of
    // 2,080 keys: 107 us with two stages and three blocks, 88 with three and two).
    static constexpr int kStages = FMT != kBF16 ? 2 : 3;
    static constexpr int CTAS = kRowBytes == 256 ? 2 : 3;
    static constexpr int kHeadWarps = kWarps / HG;               // warps of a KV head
    static constexpr int kGroup = kHeadWarps * NSUB;             // chunks of a block's step
    static constexpr int kOStride = HD + 4;                      // floats of a parked output row
    static constexpr int kRingBytes = kStages * 2 * kStepBytes;  // of one warp
    static_assert(RB * kOStride * 4 <= kRingBytes, "a warp's outputs are parked in its ring");
};

// Bits 0 .. n - 1, n clamped to 0 .. 16.
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 16 ? 0xFFFFu : (1u << n) - 1u;
}

// Byte offset of 16-byte piece c of row r (0 .. 15) of a chunk's K rows.
template <int ROW>
__device__ __forceinline__ uint32_t k_offset(int r, int c) {
    return ROW == 64 ? r * 64 + c * 16 : r * ROW + ((c ^ (4 * (r & 1))) << 4);
}

// ... of its V rows.  64-byte rows: rows 2 i and 2 i + 1 share 128 bytes, whose
// halves change places for odd i, and the 32-byte parts of a half for i & 2.
template <int ROW>
__device__ __forceinline__ uint32_t v_offset(int r, int c) {
    const int i = r >> 1;
    return ROW == 64 ? i * 128 + (((r ^ i) & 1) << 6) + ((c ^ (i & 2)) << 4)
                     : r * ROW + ((c ^ (2 * (i & 3))) << 4);
}

// 16 bytes to shared memory, asynchronously; zeros where !on.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_16_to(uint32_t dst, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// Four codes of a key -> two f16x2 words for Q K^T.  INT8: a byte with its sign
// bit flipped, c + 128, is the f16 (c + 128) 2^-24, a subnormal the tensor
// cores take exactly; the accumulators start at -128 2^-24 sum(q), so a score
// comes out as 2^-24 q . c.  (V keeps the subtraction: there the offset would
// be carried through every key's addition to O.)
constexpr uint32_t kMinus128 = 0x80808080u;  // f16x2 of -128 2^-24

template <int FMT>
__device__ __forceinline__ void key_codes_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == kINT8) {
        x ^= 0x80808080u;
        lo = __byte_perm(x, 0u, 0x4140u);
        hi = __byte_perm(x, 0u, 0x4342u);
    } else {
        codes_to_f16<FMT>(x, lo, hi);
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

// The halves of a bf16 word that are not finite.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) |
           ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}
constexpr uint32_t kOnes = 0x3F803F80u;  // bf16x2

__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int FMT>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
    if constexpr (FMT == kBF16)
        mma_bf16_16816(d, a, b0, b1);
    else
        mma_f16_16816(d, a, b0, b1);
}

// The visible keys of one (request, row block): positions [0, sinks) and
// [lo, hi); pmin, pmax the rows' first and last position.
struct Entry {
    int lo, hi, pmin, pmax;
};

// ... as chunks 0 .. sc - 1 and clo, clo + 1, ..., cnt in all.  Where the two
// ranges meet they are one, and the keys between them masked.
struct Chunks {
    int sc, clo, cnt;
};
__device__ __forceinline__ Chunks chunks_of(const Entry &t, int sinks) {
    Chunks c;
    const int chi = (t.hi + kChunk - 1) / kChunk;
    c.clo = t.lo / kChunk;
    c.sc = (min(sinks, t.hi) + kChunk - 1) / kChunk;
    if (c.sc > 0 && c.clo <= c.sc) c.clo = c.sc = 0;
    c.cnt = c.sc + chi - c.clo;
    return c;
}

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
    t.hi = max(0, (int)min((int64_t)len, (int64_t)t.pmax + 1));
    if (t.hi == 0) return t;
    t.lo = p.window > 0 ? max(0, min(t.hi, oldest - p.window + 1)) : 0;
    if (p.kind == ATTN_CACHE_RING)  // what the turning part of the ring still holds
        t.lo = max(t.lo, min(t.hi, len - (p.slots_per_seq - p.sinks)));
    if (p.from != nullptr) {
        t.lo = max(t.lo, max(0, min(p.from[b], p.from_cap)));
        if (t.lo >= t.hi) t.lo = t.hi = 0;
    }
    return t;
}

// What a warp notes about a step in its ring: whether every key of it is there,
// else the keys of each chunk that are.
template <int NSUB>
struct __align__(16) Note {
    uint32_t full, mask[NSUB];
};

template <int FMT, int HD, int MT, int HG, int ENTRIES>
struct __align__(16) Smem {
    using G = Geo<FMT, HD, MT, HG>;
    uint8_t buf[kWarps][G::kRingBytes];  // at the end of a unit a warp's output rows
    uint32_t q[HG][HD / 16][32][MT == 0 ? 2 : 4];  // q fragments of a unit, as a lane reads them
    Note<G::NSUB> note[kWarps][G::kStages];
    float m[kWarps][G::RB], l[kWarps][G::RB], w[kWarps][G::RB], lse[HG][G::RB];
    Entry entry[ENTRIES];
    int prefix[ENTRIES + 1];
    int last_part, longest;
    int share_at[2];  // the share that the CTA works on, in turn
    __device__ __forceinline__ float *out_row(int warp, int row) {
        return reinterpret_cast<float *>(buf[warp]) + row * G::kOStride;
    }
};

// The rows of a unit from its parts first .. last, by a block's four warps: rows
// warp, warp + 4, ... each, a lane HD / 32 dims of every row.  The log-sum-exps
// of 32 parts come in one load a row; the parts' outputs then wait for nothing.
template <int HD, int RB, int HG>
__device__ __forceinline__ void merge_unit(const Params &p, int64_t unit, int hs, int first,
                                           int last, int row0, int n_rows, int b, int kvh) {
    constexpr int V = HD / 32, R = RB / kWarps;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m[R], sum[R], acc[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY, sum[r] = 0.f;
#pragma unroll
        for (int d = 0; d < V; ++d) acc[r][d] = 0.f;
    }
    for (int c0 = first; c0 <= last; c0 += 32) {
        const int n = min(32, last - c0 + 1);
        float f[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = warp + kWarps * r;
            f[r] = lane < n && row < n_rows ? __ldcg(p.ws_lse + ((unit + c0 + lane) * HG + hs) * RB + row)
                                            : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float mx = f[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m[r], mx), m_use = m_new == -INFINITY ? 0.f : m_new;
            const float old = fast_exp2(m[r] - m_use);
            f[r] = kPartWeight * fast_exp2(f[r] - m_use);
            m[r] = m_new;
            sum[r] *= old;
#pragma unroll
            for (int d = 0; d < V; ++d) acc[r][d] *= fmaxf(old, kSmallest);
        }
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = min(warp + kWarps * r, n_rows - 1);
                const float w = __shfl_sync(0xffffffffu, f[r], k);
                const float *src =
                    p.ws_o + (((unit + c0 + k) * HG + hs) * RB + row) * HD + lane * V;
                sum[r] += w;
                const float wo = fmaxf(w, kSmallest);
                if constexpr (V == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
                    acc[r][0] += wo * x.x, acc[r][1] += wo * x.y;
                    acc[r][2] += wo * x.z, acc[r][3] += wo * x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
                    acc[r][0] += wo * x.x, acc[r][1] += wo * x.y;
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = warp + kWarps * r;
        if (row >= n_rows) continue;
        const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];
        const int q_row = row0 + row, qr = q_row / p.group;
        uint32_t *dst = reinterpret_cast<uint32_t *>(
            p.out + (((int64_t)b * p.q_rows + qr) * p.n_q_heads + kvh * p.group +
                     (q_row - qr * p.group)) * HD + lane * V);
#pragma unroll
        for (int d = 0; d < V / 2; ++d)
            dst[d] = pack_bf16x2(acc[r][2 * d] * inv, acc[r][2 * d + 1] * inv);
    }
}

template <int FMT, int HD, int MT, int HG, int ENTRIES>
__global__ void __launch_bounds__(kThreads, Geo<FMT, HD, MT, HG>::CTAS)
    attend_kernel(const Params p) {
    using G = Geo<FMT, HD, MT, HG>;
    constexpr int RB = G::RB;
    constexpr int kSteps = HD / 16;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using S = Smem<FMT, HD, MT, HG, ENTRIES>;
    // launch_attend_parts: shares by whoever is free, units left as parts.  Not by the parameters:
    // one request under sinks 9.46 us with the share loop in its kernel, 9.33 without
    constexpr bool kParts = ENTRIES != kMaxEntries;
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;
    if (!kParts || !p.late_wait) pdl_wait();
    pdl_launch_dependents();
    int after = (int)blockIdx.x;  // thread 0: the share that comes next
    if (kParts && threadIdx.x == 0) after = atomicAdd(p.next, 1);

    // ---- the launch's work, the same in every CTA
    for (int i = threadIdx.x; i < p.n_entries; i += kThreads)
        sm.entry[i] = make_entry(p, p.e0 + i, RB, blockIdx.x == 0);
    __syncthreads();
    if (warp == 0) {
        int carry = 0, longest = 0;
        if (lane == 0) sm.prefix[0] = 0;
        for (int base = 0; base < p.n_entries; base += 32) {
            const int i = base + lane;
            const int n = i < p.n_entries ? chunks_of(sm.entry[i], p.sinks).cnt : 0;
            longest = max(longest, n);
            int x = n > 0 ? (n + kGapChunks) * p.n_groups : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (i < p.n_entries) sm.prefix[i + 1] = carry + x;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 0) sm.longest = longest;
    }
    __syncthreads();
    const int total = sm.prefix[p.n_entries];
    int share = max(kMinChunks, (total + p.pieces - 1) / p.pieces);
    if (p.ws_count != nullptr)
        share = max(share, (sm.longest + kKernelParts - 2) / (kKernelParts - 1));

    if (blockIdx.x == 0) {
        // rows of a unit without keys are zeros, and it has no parts
        for (int i = warp; i < p.n_entries; i += kWarps) {
            if (chunks_of(sm.entry[i], p.sinks).cnt != 0) continue;
            const int e = p.e0 + i, b = e / p.row_blocks, rb = e - b * p.row_blocks;
            const int row0 = rb * RB, n = min(p.rows, row0 + RB) - row0;
            for (int kvh = 0; kvh < p.n_kv_heads; ++kvh) {
                if (lane == 0 && p.ws_count == nullptr && kvh % HG == 0)
                    p.ws_parts[i * p.n_groups + kvh / HG] = make_int2(0, -1);
                for (int j = lane; j < n * (HD / 8); j += 32) {
                    const int row = row0 + j / (HD / 8), r = row / p.group, gr = row - r * p.group;
                    reinterpret_cast<uint4 *>(
                        p.out + (((int64_t)b * p.q_rows + r) * p.n_q_heads + kvh * p.group + gr) *
                                    HD)[j % (HD / 8)] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    }

    for (int turn = 0;; turn ^= 1) {
    int piece = blockIdx.x;
    if constexpr (kParts) {
        // Two places in turn: a share that lies in a gap passes no other barrier, so one of them is
        // only written again behind the next round's, which follows every thread's read of it
        if (threadIdx.x == 0) sm.share_at[turn] = after;
        __syncthreads();
        piece = sm.share_at[turn];
        if ((int64_t)piece * share >= total) break;
        if (threadIdx.x == 0) after = atomicAdd(p.next, 1);  // (under way meanwhile)
    }
    int g = min(total, (int)min((int64_t)piece * share, (int64_t)total));
    const int g_end = min(total, g + share);
    while (g < g_end) {
        // ---- the next piece of a unit
        int lo_e = 0, hi_e = p.n_entries;
        while (hi_e - lo_e > 1) {
            const int mid = (lo_e + hi_e) >> 1;
            if (sm.prefix[mid] <= g) lo_e = mid; else hi_e = mid;
        }
        const Entry en = sm.entry[lo_e];
        const Chunks ch = chunks_of(en, p.sinks);
        const int span = ch.cnt + kGapChunks;
        int off = g - sm.prefix[lo_e];
        const int head_group = off / span;
        off -= head_group * span;
        const int hs = warp / G::kHeadWarps;        // which of the unit's heads is this warp's
        const int kvh0 = head_group * HG, kvh = kvh0 + hs;
        const int unit_start = g - off;
        if (off >= ch.cnt) {  // in the gap behind the unit
            g = unit_start + span;
            continue;
        }
        const int c_end = min(ch.cnt, off + (g_end - g));
        const int unit = lo_e * p.n_groups + head_group;
        const int first = unit_start / share, last = (unit_start + ch.cnt - 1) / share;
        const int e = p.e0 + lo_e, b = e / p.row_blocks, rb = e - b * p.row_blocks;
        const int row0 = rb * RB, n_rows = min(p.rows, row0 + RB) - row0;

        // ---- q rows
        const __nv_bfloat16 *qb =
            p.q + ((int64_t)b * p.q_rows * p.n_q_heads + kvh0 * p.group) * HD;
        auto row_of = [&](int rr) {  // row rr of the unit, in q and out
            const int row = row0 + min(rr, n_rows - 1), r = row / p.group;
            return ((int64_t)r * p.n_q_heads + (row - r * p.group)) * HD;
        };
        auto pos_of = [&](int rr) {
            return p.positions[(int64_t)b * p.q_rows + (row0 + min(rr, n_rows - 1)) / p.group];
        };
        // the row (0 or 1 of the thread's two) of accumulator element e
        auto row_e = [](int e) { return MT == 0 ? (e & 1) : (e >> 1); };

        // ---- where chunks lie
        constexpr int NSUB = G::NSUB;
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
        auto real_chunk = [&](int c) { return c < ch.sc ? c : c - ch.sc + ch.clo; };
        auto chunk_mask = [&](int t0) -> uint32_t {
            return (bits_below(p.sinks - t0) | (0xFFFFu & ~bits_below(en.lo - t0))) &
                   bits_below(en.hi - t0);
        };
        auto page_of_chunk = [&](int rc) {
            return (int)(__umulhi((uint32_t)rc << 4, p.page_mul) >> p.page_shift);
        };
        // What is the same for a whole chunk is worked out by one lane for 32 chunks at a
        // time (kAhead steps: lane l has chunk l % NSUB of step l / NSUB) and handed out by
        // shuffles; the table entries are read kAhead steps before that.
        constexpr int kAhead = 32 / NSUB;
        auto chunk_of_lane = [&](int c) { return c + lane / NSUB * G::kGroup + lane % NSUB; };
        int page = 0;
        auto read_pages = [&](int c) {
            const int cc = chunk_of_lane(c);
            if (p.kind == ATTN_CACHE_PAGED && even && cc < c_end)
                page = __ldg(bt + page_of_chunk(real_chunk(cc)));
        };

        float o[MT == 0 ? HD / 16 : HD / 8][4];
        float m_run[2], l_run[2];

        // ---- copies of a step's keys
        constexpr int kPer = G::kRowBytes / 16;  // 16-byte pieces of a row
        constexpr int kRowsPer = 32 / kPer;      // rows of one copy instruction
        const int my_row = lane / kPer, my_piece = lane % kPer;
        const uint32_t ring = smem_u32(sm.buf[warp]);
        // this lane's first piece of an evenly spaced chunk, and from one to the next
        const uint32_t lane_at = my_row * row_step * G::kRowBytes + my_piece * 16;
        const uint8_t *const k_lane = p.k + lane_at, *const v_lane = p.v + lane_at;
        const uint32_t k_to = k_offset<G::kRowBytes>(my_row, my_piece);
        const uint32_t v_to = v_offset<G::kRowBytes>(my_row, my_piece);
        // where this thread reads its share of K and V in a chunk
        const uint32_t k_from = k_offset<G::kRowBytes>(gq, tq);
        const uint32_t v_from = G::kVBytes == 8
                                    ? v_offset<G::kRowBytes>(2 * tq, gq >> 1) + 8 * (gq & 1)
                                    : v_offset<G::kRowBytes>(2 * tq, gq);
        // where position t of a ring lies in it
        auto ring_row = [&](int t) {
            return t < p.sinks ? t : p.sinks + (t - p.sinks) % (p.slots_per_seq - p.sinks);
        };
        // For steps c .. c + (kAhead - 1) kGroup: each chunk's first row, whether it is
        // there (a page outside the pool is reported), whether all its keys are visible
        // and evenly spaced, and its scales
        uint32_t top = 0, there = 0, entire = 0;
        float next_sk = 1.f, next_sv = 1.f;
        auto locate = [&](int c) {
            const int cc = chunk_of_lane(c), rc = real_chunk(cc), t0 = rc * kChunk;
            bool good = cc < c_end, run = even;
            int slot = 0;
            top = 0;
            next_sk = next_sv = 1.f;
            if (good) {
                if (p.kind == ATTN_CACHE_RING) {
                    const int r = ring_row(t0);
                    top = row_index(b, r);
                    run = t0 + kChunk <= p.sinks || (t0 >= p.sinks && r + kChunk <= p.slots_per_seq);
                } else if (p.kind != ATTN_CACHE_PAGED) {
                    top = row_index(b, t0);
                    slot = b * p.slots_per_seq + t0;
                } else if (even) {
                    good = (unsigned)page < (unsigned)p.num_pages;
                    if (good) {
                        const int r = (rc - page_of_chunk(rc) * p.page_chunks) * kChunk;
                        top = row_index(page, r);
                        slot = page * p.block_size + r;
                    } else {
                        report_error(p.err, ATTN_ERR_BOUNDS);
                    }
                }
            }
            there = __ballot_sync(0xffffffffu, good);
            entire = __ballot_sync(0xffffffffu, good && run && chunk_mask(t0) == 0xFFFFu);
            if constexpr (FMT != kBF16)
                if (p.ks != nullptr && good) {
                    const int64_t at = (int64_t)(slot >> p.scale_shift) * p.n_kv_heads + kvh;
                    next_sk = __ldg(p.ks + at);
                    next_sv = __ldg(p.vs + at);
                }
        };
        // requests step c (nothing past c_end), the k-th located, into stage st
        auto request = [&](int c, int k, int st) {
            const uint32_t k_buf = ring + st * 2 * G::kStepBytes, v_buf = k_buf + G::kStepBytes;
            Note<NSUB> &note = sm.note[warp][st];
            const uint32_t all = ((1u << NSUB) - 1u) << (k * NSUB);
            const bool full = (entire & all) == all && (c >= ch.sc || c + NSUB <= ch.sc);
            if (full) {
#pragma unroll
                for (int i = 0; i < NSUB; ++i) {
                    uint32_t row = __shfl_sync(0xffffffffu, top, k * NSUB + i);
#pragma unroll
                    for (int n = 0; n < kChunk / kRowsPer; ++n) {
                        // v_offset of row my_row + n kRowsPer against my_row's
                        const int flip = G::kRowBytes == 128   ? 64 * (n & 1)
                                         : G::kRowBytes == 256 ? 32 * (n & 3)
                                                               : 0;
                        const int to = i * G::kChunkBytes + n * 512;
                        const uint64_t at = (uint64_t)row * G::kRowBytes;
                        cp_async_16_to(k_buf + k_to + to, k_lane + at);
                        cp_async_16_to(v_buf + (v_to ^ flip) + to, v_lane + at);
                        row += kRowsPer * row_step;
                    }
                }
            }
            if (lane == 0) note.full = full;
            if (!full) {
                // key by key; keys that are absent become zeros
#pragma unroll
                for (int i = 0; i < NSUB; ++i) {
                    const int rc = real_chunk(c + i), t = rc * kChunk + (lane & 15);
                    const uint32_t first = __shfl_sync(0xffffffffu, top, k * NSUB + i);
                    uint32_t mask = (there >> (k * NSUB + i)) & 1u ? chunk_mask(rc * kChunk) : 0u;
                    uint32_t spread = 0;
                    if (!even) {
                        bool on = (mask >> (lane & 15)) & 1u;
                        if (on && p.kind == ATTN_CACHE_PAGED) {
                            const int pi = t / p.block_size, id = __ldg(bt + pi);
                            if ((unsigned)id >= (unsigned)p.num_pages) {
                                report_error(p.err, ATTN_ERR_BOUNDS);
                                on = false;
                            } else {
                                spread = row_index(id, t - pi * p.block_size);
                            }
                        } else if (on) {
                            spread = row_index(b, ring_row(t));
                        }
                        mask = __ballot_sync(0xffffffffu, on) & 0xFFFFu;
                    }
                    if (lane == 0) note.mask[i] = mask;
#pragma unroll
                    for (int n = 0; n < kChunk / kRowsPer; ++n) {
                        const int r = my_row + n * kRowsPer;
                        const uint32_t row = even ? first + r * row_step
                                                  : __shfl_sync(0xffffffffu, spread, r);
                        const bool on = (mask >> r) & 1u;
                        const uint64_t at =
                            on ? (uint64_t)row * G::kRowBytes + my_piece * 16 : (uint64_t)0;
                        const int to = i * G::kChunkBytes;
                        copy16(k_buf + to + k_offset<G::kRowBytes>(r, my_piece), p.k + at, on);
                        copy16(v_buf + to + v_offset<G::kRowBytes>(r, my_piece), p.v + at, on);
                    }
                }
            }
        };

        const int c0 = off + warp % G::kHeadWarps * NSUB;
        constexpr int kQRows = MT == 0 ? 1 : 2;
        int rpos[2];  // positions of the two rows this thread keeps scores of
        float q_bias[2] = {0.f, 0.f};  // -128 2^-24 sum(q) of the two rows
        // q fragments and positions are asked for before the keys, or they would come behind them
        // (64 requests x 4 rows of 64 to 4,096 INT8 keys 59.1 us, after the first keys 60.0; one
        // request of 512 E4M3 keys 7.35 and 7.22, 16 x 32 heads of 64 the same)
        constexpr int kMine = (HG * kSteps + kWarps - 1) / kWarps;
        uint2 q_in[kMine][kQRows];
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
            const int i = warp + n * kWarps, qs = i / kSteps, kk = i % kSteps;  // head, k-step
            const int j = kk / G::kStepsPerPiece, st = kk % G::kStepsPerPiece;
            const int d0 = (16 / G::E) * (tq + 4 * j) + 4 * st;
            if (i < HG * kSteps)
#pragma unroll
                for (int hr = 0; hr < kQRows; ++hr)
                    q_in[n][hr] = *reinterpret_cast<const uint2 *>(qb + qs * p.group * HD +
                                                                   row_of(gq + 8 * hr) + d0);
        }
        rpos[0] = MT == 0 ? pos_of(2 * tq) : pos_of(gq);
        rpos[1] = MT == 0 ? pos_of(2 * tq + 1) : pos_of(gq + 8);
        // This warp's chunks; bf16 again where an infinity in V may have become a NaN (by the
        // lower half of its weight, which may be 0 or negative, or by a factor that is 0)
        for (bool again = false;; again = true) {
#pragma unroll
            for (auto &x : o) x[0] = x[1] = x[2] = x[3] = 0.f;
            m_run[0] = m_run[1] = -INFINITY, l_run[0] = l_run[1] = 0.f;
            read_pages(c0);
            locate(c0);
            read_pages(c0 + kAhead * G::kGroup);
#pragma unroll
            for (int st = 0; st < G::kStages - 1; ++st) {
                const int c = c0 + st * G::kGroup;
                if (c < c_end) request(c, st, st);
                copies_commit();
            }
            if (!again) {
                bool q_big = false;
#pragma unroll
                for (int n = 0; n < kMine; ++n) {
                    const int i = warp + n * kWarps, qs = i / kSteps, kk = i % kSteps;
                    if (i >= HG * kSteps) break;
#pragma unroll
                    for (int hr = 0; hr < kQRows; ++hr) {
                        uint2 x = q_in[n][hr];
                        if constexpr (FMT != kBF16) {  // f16 holds |q| < 65520
                            x.x = bf16x2_to_f16x2(x.x);
                            x.y = bf16x2_to_f16x2(x.y);
                            q_big |= (x.x & 0x7C00u) == 0x7C00u || (x.x & 0x7C000000u) == 0x7C000000u ||
                                     (x.y & 0x7C00u) == 0x7C00u || (x.y & 0x7C000000u) == 0x7C000000u;
                        }
                        sm.q[qs][kk][lane][hr] = x.x;
                        sm.q[qs][kk][lane][kQRows + hr] = x.y;
                    }
                }
                if (q_big) report_error(p.err, ATTN_ERR_UNSUPPORTED);
                __syncthreads();

                if constexpr (FMT == kINT8) {
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    const uint32_t a[4] = {kMinus128, kMinus128, kMinus128, kMinus128};
#pragma unroll
                    for (int kk = 0; kk < kSteps; ++kk) {
                        if constexpr (MT == 0) {
                            mma_f16_16816(sum, a, sm.q[hs][kk][lane][0], sm.q[hs][kk][lane][1]);
                        } else {
                            const uint32_t qa[4] = {sm.q[hs][kk][lane][0], sm.q[hs][kk][lane][1],
                                                    sm.q[hs][kk][lane][2], sm.q[hs][kk][lane][3]};
                            mma_f16_16816(sum, qa, kMinus128, kMinus128);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) q_bias[row_e(e)] = sum[e];
                }
            }
            // of 32 chunks, a lane each: what scores are multiplied with, log2 and inverse of V's scale
            float f_lane = p.scale_log2, lv_lane = 0.f, inv_lane = 1.f;
            int st = 0, step = 0;
            for (int c = c0; c < c_end; c += G::kGroup, ++step, st = st + 1 == G::kStages ? 0 : st + 1) {
                copies_wait<G::kStages - 2>();
                __syncwarp();  // the step has landed for all lanes, and the step before is read
                const int ahead = c + (G::kStages - 1) * G::kGroup;
                if (ahead < c_end) {
                    const int k = (step + G::kStages - 1) % kAhead;
                    if (k == 0) {
                        locate(ahead);
                        read_pages(ahead + kAhead * G::kGroup);
                    }
                    request(ahead, k, st == 0 ? G::kStages - 1 : st - 1);
                }
                copies_commit();
                const int of_step = step % kAhead * NSUB;  // the lane that has the step's first chunk
                if (FMT != kBF16 && of_step == 0) {
                    const float sv = fmaxf(next_sv, kScaleFloor);
                    f_lane = fmaxf(next_sk, kScaleFloor) *
                             (FMT == kINT8 ? p.scale_log2 * 16777216.f : p.scale_log2);
                    f_lane = fminf(f_lane, kFactorTop);
                    lv_lane = fast_log2(sv);
                    inv_lane = 0.25f * fast_rcp(0.25f * sv);  // subnormal from 2^126 on, not 0
                }
                const uint32_t k_buf = ring + st * 2 * G::kStepBytes, v_buf = k_buf + G::kStepBytes;
                const Note<NSUB> &note = sm.note[warp][st];
                const bool cur_full = note.full != 0;
                uint32_t kw[NSUB][2][4 * G::kKPieces];
#pragma unroll
                for (int i = 0; i < NSUB; ++i) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < G::kKPieces; ++j) {
                            // piece tq + 4 j of row gq + 8 h
                            const uint4 x = ld_shared_v4(k_buf + i * G::kChunkBytes +
                                                         8 * h * G::kRowBytes +
                                                         (k_from ^ (64 * (j & 1))) + 128 * (j >> 1));
                            kw[i][h][4 * j] = x.x, kw[i][h][4 * j + 1] = x.y;
                            kw[i][h][4 * j + 2] = x.z, kw[i][h][4 * j + 3] = x.w;
                        }
                }
                // ---- scores: MT 0 keys are the rows of S^T = K Q^T, MT 1 the columns of S = Q K^T.
                // Even and odd k-steps add up apart: a product waits for half as many before it
                constexpr int NJ = MT == 0 ? 1 : 2;
                float s[NSUB][NJ][4];
                float s_odd[NSUB][NJ][4];
#pragma unroll
                for (int i = 0; i < NSUB; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[i][j][e] = FMT == kINT8 ? q_bias[row_e(e)] : 0.f;
                            s_odd[i][j][e] = 0.f;
                        }
#pragma unroll
                for (int kk = 0; kk < kSteps; ++kk) {
                    uint32_t qf[2 * kQRows];
                    if constexpr (MT == 0) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(sm.q[hs][kk][lane]);
                        qf[0] = x.x, qf[1] = x.y;
                    } else {
                        const uint4 x = *reinterpret_cast<const uint4 *>(sm.q[hs][kk][lane]);
                        qf[0] = x.x, qf[1] = x.y, qf[2] = x.z, qf[3] = x.w;
                    }
#pragma unroll
                    for (int i = 0; i < NSUB; ++i) {
                        uint32_t x[2][2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if constexpr (FMT == kBF16) {
                                x[h][0] = kw[i][h][2 * kk];
                                x[h][1] = kw[i][h][2 * kk + 1];
                            } else {
                                key_codes_to_f16<FMT>(kw[i][h][kk], x[h][0], x[h][1]);
                            }
                        }
                        if constexpr (MT == 0) {
                            const uint32_t a[4] = {x[0][0], x[1][0], x[0][1], x[1][1]};
                            mma16<FMT>(kk & 1 ? s_odd[i][0] : s[i][0], a, qf[0], qf[1]);
                        } else {
                            mma16<FMT>(s[i][0], qf, x[0][0], x[0][1]);
                            mma16<FMT>(s[i][1], qf, x[1][0], x[1][1]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < NSUB; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if constexpr (MT == 0) s[i][j][e] += s_odd[i][j][e];
                // ---- mask and weights.  x(row, key): element e of s[i][j] is
                // MT 0: row e & 1, key gq + 8 (e >> 1); MT 1: row e >> 1, key 8 j + 2 tq + (e & 1)
                auto sees = [&](int i, int row, int key) {
                    const int t = real_chunk(c + i) * kChunk + key, pos = rpos[row];
                    return (cur_full || ((note.mask[i] >> key) & 1u)) && t <= pos &&
                           (p.window <= 0 || pos - t < p.window || t < p.sinks);
                };
                float f[NSUB], lv[NSUB], inv_sv[NSUB];
                const int first_t = real_chunk(c) * kChunk, end_t = first_t + NSUB * kChunk;
                // every row sees every key of the step
                const bool open = cur_full && !(FMT == kBF16 && again) && end_t - 1 <= en.pmin &&
                                  (p.window <= 0 || en.pmax - first_t < p.window || end_t <= p.sinks);
#pragma unroll
                for (int i = 0; i < NSUB; ++i) {
                    f[i] = FMT == kBF16 ? f_lane : __shfl_sync(0xffffffffu, f_lane, of_step + i);
                    lv[i] = FMT == kBF16 ? 0.f : __shfl_sync(0xffffffffu, lv_lane, of_step + i);
                    inv_sv[i] = FMT == kBF16 ? 1.f : __shfl_sync(0xffffffffu, inv_lane, of_step + i);
                }
                if (!open) {
#pragma unroll
                    for (int i = 0; i < NSUB; ++i)
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = MT == 0 ? gq + 8 * (e >> 1) : 8 * j + 2 * tq + (e & 1);
                                s[i][j][e] = sees(i, row_e(e), key) ? s[i][j][e] : -INFINITY;
                            }
                }
                float alpha[2];
                bool moved = false;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    // x = s f + lv grows with s (f > 0): its maximum is that of s
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NSUB; ++i) {
                        float ms = fmaxf(s[i][0][MT == 0 ? r : 2 * r], s[i][0][MT == 0 ? r + 2 : 2 * r + 1]);
                        if constexpr (NJ > 1) ms = max3(ms, s[i][1][2 * r], s[i][1][2 * r + 1]);
                        mx = fmaxf(mx, fmaf(ms, f[i], lv[i]));
                    }
                    if constexpr (MT == 0) {
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    } else {
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    }
                    const float m_old = m_run[r];
                    const float m_new = mx > m_old + kRescaleLog2 ? mx : m_old;
                    const float m_use = m_new == -INFINITY ? 0.f : m_new;
                    const float m_w = FMT == kBF16 ? m_use : m_use - kWeightLog2;
                    alpha[r] = m_new == m_old ? 1.f : fast_exp2(m_old - m_use);
                    moved |= m_new != m_old;
                    m_run[r] = m_new;
                    l_run[r] *= alpha[r];
#pragma unroll
                    for (int i = 0; i < NSUB; ++i) {
                        const float shift = lv[i] - m_w;
                        float sum = 0.f;
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (row_e(e) == r) {
                                    s[i][j][e] = fast_exp2(fmaf(s[i][j][e], f[i], shift));
                                    sum += s[i][j][e];
                                }
                        l_run[r] = fmaf(sum, inv_sv[i], l_run[r]);
                    }
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (auto &x : o)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] *= FMT == kBF16 ? fmaxf(alpha[row_e(e)], kSmallest)
                                                 : alpha[row_e(e)];
                }
                // ---- P V, a chunk at a time.  Weights as its operand: f16 (one rounding:
                // 11 bits), or for a bf16 cache two bf16 halves (16 bits), since one
                // bf16 rounding of P would cost as much as the output's own
                constexpr int NP = MT == 0 ? 2 : 4;
                constexpr int kPairs = HD / 16;            // pairs of dims of a thread
                constexpr int kPairsPerWord = 2 / G::E;
#pragma unroll
                for (int i = 0; i < NSUB; ++i) {
                    uint32_t ph[NP], pl[NP];
                    if constexpr (MT == 0) {
                        if constexpr (FMT == kBF16) {
                            split_bf16x2(s[i][0][0], s[i][0][1], ph[0], pl[0]);
                            split_bf16x2(s[i][0][2], s[i][0][3], ph[1], pl[1]);
                            pl[0] = movmatrix_trans(pl[0]);
                            pl[1] = movmatrix_trans(pl[1]);
                        } else {
                            ph[0] = pack_f16x2(s[i][0][0], s[i][0][1]);
                            ph[1] = pack_f16x2(s[i][0][2], s[i][0][3]);
                        }
                        ph[0] = movmatrix_trans(ph[0]);
                        ph[1] = movmatrix_trans(ph[1]);
                    } else {
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const int j = n >> 1, r = n & 1;
                            if constexpr (FMT == kBF16)
                                split_bf16x2(s[i][j][2 * r], s[i][j][2 * r + 1], ph[n], pl[n]);
                            else
                                ph[n] = pack_f16x2(s[i][j][2 * r], s[i][j][2 * r + 1]);
                        }
                    }
                    // V operands of two neighbouring dims (word w of a thread's share): x[0]
                    // and x[1] dim 0 and 1 over keys 2 tq, 2 tq + 1, x[2] and x[3] over + 8
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
                    auto add_pv = [&](const uint32_t (&x)[4], float (&oa)[4], float (&ob)[4]) {
                        if constexpr (MT == 0) {  // O^T: dim 0 in elements 0, 1, dim 1 in 2, 3
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
                    uint32_t vw[4][G::kVWords];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint32_t src =
                            v_buf + i * G::kChunkBytes + 8 * (n >> 1) * G::kRowBytes;
                        if constexpr (G::kVBytes == 8) {
                            const uint2 x = ld_shared_v2(src + (v_from ^ (64 * (n & 1))));
                            vw[n][0] = x.x, vw[n][1] = x.y;
                        } else {
#pragma unroll
                            for (int j = 0; j < G::kVPieces; ++j) {
                                const uint4 x =
                                    ld_shared_v4(src + v_from + (n & 1) * G::kRowBytes + 128 * j);
                                vw[n][4 * j] = x.x, vw[n][4 * j + 1] = x.y;
                                vw[n][4 * j + 2] = x.z, vw[n][4 * j + 3] = x.w;
                            }
                        }
                    }
                    if constexpr (FMT != kINT8) {
                        if (!open) {
                            // A value that is not finite reaches only the rows that see its
                            // key: 0 times it would be NaN in every row.  Such keys are
                            // multiplied alone, added where seen, and taken out (bf16: such
                            // values, and by 1: any weight above 0 gives the same).
                            uint32_t odd = 0;
#pragma unroll
                            for (int n = 0; n < 4; ++n)
#pragma unroll
                                for (int w = 0; w < G::kVWords; ++w)
                                    if (word_not_finite<FMT>(vw[n][w]))
                                        odd |= 1u << (2 * tq + (n & 1) + 8 * (n >> 1));
                            odd = __reduce_or_sync(0xffffffffu, odd);
                            while (odd != 0) {
                                const int key = __ffs(odd) - 1;
                                odd &= odd - 1;
#pragma unroll
                                for (int d = 0; d < kPairs; ++d) {
                                    uint32_t w[4], x[4];
#pragma unroll
                                    for (int n = 0; n < 4; ++n) {
                                        uint32_t &v = vw[n][d / kPairsPerWord];
                                        const bool its = key == 2 * tq + (n & 1) + 8 * (n >> 1);
                                        w[n] = !its ? 0u : FMT == kBF16 ? v & odd_halves(v) : v;
                                        if (FMT == kBF16 && its) v &= ~odd_halves(v);
                                    }
                                    v_pair(w, d % kPairsPerWord, x);
                                    float ta[4] = {0.f, 0.f, 0.f, 0.f}, tb[4] = {0.f, 0.f, 0.f, 0.f};
                                    if constexpr (FMT != kBF16) {
                                        add_pv(x, ta, tb);
                                    } else if constexpr (MT == 0) {
                                        mma16<FMT>(ta, x, kOnes, kOnes);
                                    } else {
                                        const uint32_t ones[4] = {kOnes, kOnes, kOnes, kOnes};
                                        mma16<FMT>(ta, ones, x[0], x[2]);
                                        mma16<FMT>(tb, ones, x[1], x[3]);
                                    }
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (sees(i, row_e(e), key)) {
                                            o[MT == 0 ? d : 2 * d][e] += ta[e];
                                            if constexpr (MT != 0) o[2 * d + 1][e] += tb[e];
                                        }
                                }
#pragma unroll
                                for (int n = 0; n < 4; ++n)
                                    if (FMT != kBF16 && key == 2 * tq + (n & 1) + 8 * (n >> 1))
#pragma unroll
                                        for (int w = 0; w < G::kVWords; ++w) vw[n][w] = 0u;
                            }
                        }
                    }
#pragma unroll
                    for (int d = 0; d < kPairs; ++d) {
                        uint32_t w[4], x[4];
#pragma unroll
                        for (int n = 0; n < 4; ++n) w[n] = vw[n][d / kPairsPerWord];
                        v_pair(w, d % kPairsPerWord, x);
                        if constexpr (MT == 0)
                            add_pv(x, o[d], o[d]);
                        else
                            add_pv(x, o[2 * d], o[2 * d + 1]);
                    }
                }
            }
            copies_wait<0>();
            __syncwarp();  // the ring is this warp's to write
            if constexpr (FMT != kBF16) break;
            bool nan = false;
#pragma unroll
            for (auto &x : o) nan |= isnan(x[0]) || isnan(x[1]) || isnan(x[2]) || isnan(x[3]);
            if (again || !__any_sync(0xffffffffu, nan)) break;
        }
        // (-inf: no key seen)
        if (fmaxf(m_run[0] == -INFINITY ? 0.f : fabsf(m_run[0]),
                  m_run[1] == -INFINITY ? 0.f : fabsf(m_run[1])) >=
            (FMT == kBF16 ? kScoreTopBf16 : kScoreTopF16))
            report_error(p.err, ATTN_ERR_UNSUPPORTED);

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
        // dim d (0 .. HD / 8 - 1) of a thread group
        auto dim_of = [](int g8, int d) {
            return G::kVElems * (g8 + 8 * (d / G::kVElems)) + d % G::kVElems;
        };
        if constexpr (MT == 0) {
#pragma unroll
            for (int d = 0; d < HD / 16; ++d)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    *reinterpret_cast<float2 *>(sm.out_row(warp, 2 * tq + r) + dim_of(gq, 2 * d)) =
                        make_float2(o[d][r], o[d][r + 2]);
        } else {
#pragma unroll
            for (int d = 0; d < HD / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float2 *>(sm.out_row(warp, gq + 8 * (i >> 1)) +
                                                dim_of(2 * tq + (i & 1), 2 * d)) =
                        make_float2(o[2 * d][i], o[2 * d + 1][i]);
        }
        __syncthreads();
        if (threadIdx.x < HG * RB) {
            constexpr int W = G::kHeadWarps;
            const int row = threadIdx.x % RB, h = threadIdx.x / RB, w0 = h * W;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) m = fmaxf(m, sm.m[w0 + w][row]);
            const float m_use = m == -INFINITY ? 0.f : m;
            float f[W];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                f[w] = fast_exp2(sm.m[w0 + w][row] - m_use);
                l += f[w] * sm.l[w0 + w][row];
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int w = 0; w < W; ++w)
                sm.w[w0 + w][row] = FMT == kBF16 ? fmaxf(f[w] * inv, kSmallest) : f[w] * inv;
            sm.lse[h][row] = l == 0.f ? -INFINITY : m_use + log2f(l);
        }
        __syncthreads();
        const bool whole = !kParts && first == last;
        const int64_t slot = (int64_t)(unit + piece) * HG;  // unique: shares are contiguous
        for (int i = threadIdx.x; i < HG * n_rows * (HD / 4); i += kThreads) {
            const int hr = i / (HD / 4), d = (i % (HD / 4)) * 4;
            const int h = HG == 1 ? 0 : hr / n_rows, row = hr - h * n_rows;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < G::kHeadWarps; ++w) {
                const int wi = h * G::kHeadWarps + w;
                const float4 x = *reinterpret_cast<const float4 *>(sm.out_row(wi, row) + d);
                const float f = sm.w[wi][row];
                a.x += f * x.x, a.y += f * x.y, a.z += f * x.z, a.w += f * x.w;
            }
            if (whole) {
                uint2 y;
                y.x = pack_bf16x2(a.x, a.y);
                y.y = pack_bf16x2(a.z, a.w);
                *reinterpret_cast<uint2 *>(
                    p.out +
                    ((int64_t)b * p.q_rows * p.n_q_heads + (kvh0 + h) * p.group) * HD +
                    row_of(row) + d) = y;
            } else {
                *reinterpret_cast<float4 *>(p.ws_o + ((slot + h) * RB + row) * HD + d) = a;
            }
        }
        if (!whole && threadIdx.x < HG * RB && threadIdx.x % RB < n_rows)
            p.ws_lse[slot * RB + threadIdx.x] = sm.lse[threadIdx.x / RB][threadIdx.x % RB];
        if (p.ws_count == nullptr) {
            if (off == 0 && threadIdx.x == 0) p.ws_parts[unit] = make_int2(first, last);
        } else if (!whole) {
            // the block that stores a unit's last part adds them all, in order
            __syncthreads();
            if (threadIdx.x == 0) {
                const bool mine = atom_add_acq_rel_gpu(p.ws_count + unit, 1) == last - first;
                if (mine) p.ws_count[unit] = 0;
                sm.last_part = mine;
            }
            __syncthreads();
            if (sm.last_part)
                for (int h = 0; h < HG; ++h)
                    merge_unit<HD, RB, HG>(p, unit, h, first, last, row0, n_rows, b, kvh0 + h);
        }
        __syncthreads();  // the shared states are free again
        g += c_end - off;
    }
    if constexpr (!kParts) break;
    }
    if (kParts && p.late_wait) pdl_wait();
}

// Adds the partial states of every unit that more than one CTA held, in part
// order within a warp and in warp order across them.  A row of a unit is read
// by SPLIT warps, each every SPLIT-th part, its lanes along the head; all of a
// warp's log-sum-exps come in one load a 32 parts, so its reads of the partial
// outputs wait for nothing but that.
template <int HD, int RB, int HG, int SPLIT>
__global__ void __launch_bounds__(256) attend_merge_kernel(const Params p) {
    constexpr int V = HD / 32;           // dims of a lane
    constexpr int kRows = 8 / SPLIT;     // rows of a block
    __shared__ float sm_acc[8][HD];
    __shared__ float sm_m[8], sm_sum[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * kRows + warp / SPLIT;
    const int64_t head = i / RB;  // KV heads of all entries
    const int row = (int)(i - head * RB);
    const int entry = (int)(head / p.n_kv_heads), kvh = (int)(head - (int64_t)entry * p.n_kv_heads);
    const int64_t unit = head / HG;
    const int hs = (int)(head - unit * HG);
    const int e = p.e0 + entry, b = e / p.row_blocks, rb = e - b * p.row_blocks;
    const int q_row = rb * RB + row;
    pdl_wait();
    pdl_launch_dependents();
    int2 parts = make_int2(0, -1);
    if (entry < p.n_entries && q_row < p.rows) parts = p.ws_parts[unit];
    const bool live = parts.y > parts.x;
    if (SPLIT == 1 && !live) return;
    float m = -INFINITY, sum = 0.f, acc[V] = {};
    if (live) {
        for (int c0 = parts.x + warp % SPLIT; c0 <= parts.y; c0 += 32 * SPLIT) {
            const int mine = c0 + lane * SPLIT;
            const float lse = mine <= parts.y ? __ldcg(p.ws_lse + ((unit + mine) * HG + hs) * RB + row)
                                               : -INFINITY;
            float mx = lse;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m, mx), m_use = m_new == -INFINITY ? 0.f : m_new;
            const float old = m == -INFINITY ? 0.f : fast_exp2(m - m_use);
            const float f = kPartWeight * fast_exp2(lse - m_use);
            m = m_new;
            sum *= old;
#pragma unroll
            for (int d = 0; d < V; ++d) acc[d] *= fmaxf(old, kSmallest);
            const int n = min(32, (parts.y - c0) / SPLIT + 1);
            const float *src = p.ws_o + (((unit + c0) * HG + hs) * RB + row) * HD + lane * V;
#pragma unroll 8
            for (int k = 0; k < n; ++k, src += (int64_t)SPLIT * HG * RB * HD) {
                const float w = __shfl_sync(0xffffffffu, f, k);
                sum += w;
                const float wo = fmaxf(w, kSmallest);
                if constexpr (V == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
                    acc[0] += wo * x.x, acc[1] += wo * x.y, acc[2] += wo * x.z, acc[3] += wo * x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
                    acc[0] += wo * x.x, acc[1] += wo * x.y;
                }
            }
        }
    }
    if constexpr (SPLIT > 1) {
#pragma unroll
        for (int d = 0; d < V; ++d) sm_acc[warp][lane * V + d] = acc[d];
        if (lane == 0) sm_m[warp] = m, sm_sum[warp] = sum;
        __syncthreads();
        if (warp % SPLIT != 0 || !live) return;
        for (int w = warp + 1; w < warp + SPLIT; ++w) {
            const float m_new = fmaxf(m, sm_m[w]), m_use = m_new == -INFINITY ? 0.f : m_new;
            const float fa = fast_exp2(m - m_use), fb = fast_exp2(sm_m[w] - m_use);
            m = m_new;
            sum = sum * fa + sm_sum[w] * fb;
#pragma unroll
            for (int d = 0; d < V; ++d)
                acc[d] = acc[d] * fmaxf(fa, kSmallest) + sm_acc[w][lane * V + d] * fmaxf(fb, kSmallest);
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

template <int FMT, int HD, int MT, int HG, int ENTRIES = kMaxEntries>
int launch(const Params &p, bool merge, cudaStream_t stream) {
    constexpr int RB = MT == 0 ? 8 : 16;
    constexpr size_t kBytes = sizeof(Smem<FMT, HD, MT, HG, ENTRIES>);
    auto kernel = attend_kernel<FMT, HD, MT, HG, ENTRIES>;
    static std::atomic<uint64_t> configured{0};  // a bit per device
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(configured.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes);
        if (e != cudaSuccess) {
            note_cuda_error(e);
            return ATTN_ERR_CUDA;
        }
        configured.fetch_or(bit, std::memory_order_relaxed);
    }
    const cudaError_t e0 =
        launch_pdl(kernel, dim3((unsigned)p.grid), dim3(kThreads), kBytes, stream, p);
    if (e0 != cudaSuccess) return ATTN_ERR_CUDA;
    if constexpr (ENTRIES != kMaxEntries) return ATTN_OK;  // (its merge is the caller's)
    if (!merge) return ATTN_OK;
    // Units that lie in many parts (few units, long contexts) have eight warps a row
    const int64_t units = (int64_t)p.n_entries * p.n_groups, rows = units * HG * RB;
    const cudaError_t e =
        p.grid > 8 * units
            ? launch_pdl(attend_merge_kernel<HD, RB, HG, 8>, dim3((unsigned)rows), dim3(256), 0, stream, p)
            : launch_pdl(attend_merge_kernel<HD, RB, HG, 1>, dim3((unsigned)((rows + 7) / 8)), dim3(256),
                         0, stream, p);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace att

// KV heads of a unit of launch_attend_parts.  Short stretches of own keys are many units of few
// chunks, whose cost is the round trips of a change of unit; heads together share them.  A step of
// attn_decode_shared, 64 bf16 requests of 64 to 1,024 own keys, 32/8 x 128: 47.8 us with four heads,
// 53.1 with two, 48.2 with one; 256 of 32 to 256: 155, 164 and 181.  8-bit rows of 128 dims (registers
// for two only): 123 E4M3 requests of 16 to 700 keys 61.3 with two, 89 with one.
static int part_heads(const attn_kv_cache *cache, int mt, int n_kv_heads, int head_dim) {
    const int most = (cache->dtype == ATTN_KV_BF16 || head_dim == 64) && mt == 0 ? 4 : 2;
    return n_kv_heads % most == 0 ? most : n_kv_heads % 2 == 0 ? 2 : 1;
}

int plan_attend(const attn_kv_cache *cache, int batch, int q_rows, int n_q_heads, int n_kv_heads,
                int head_dim, int max_seq_len, int window, int sinks, AttendPlan *plan,
                bool parts) {
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
    // Two KV heads a unit where the slot-major rows of a head are so short that one
    // head alone reads DRAM badly: 8-bit rows of 64 bytes leave half of every line
    // (16 x 32 heads, 2,048 to 8,192 keys: 595 MB from DRAM and 102 us, with two heads
    // 71 us), and bf16 rows of 128 bytes at up to 8 query rows (16 x 32 heads of 5,120
    // keys 117 us, 107 with two).  8-bit rows of 128 bytes are better alone (64 x 8
    // heads of 2,080 keys 53 us, 55 with two), as are four heads of 64 bytes (75 us).
    plan->heads = 1;
    if (cache->layout == ATTN_LAYOUT_BSHD && head_dim == 64 && n_kv_heads % 2 == 0 &&
        (cache->dtype != ATTN_KV_BF16 || plan->mt == 0))
        plan->heads = 2;
    if (parts) plan->heads = part_heads(cache, plan->mt, n_kv_heads, head_dim);
    const int n_groups = n_kv_heads / plan->heads;
    const int64_t per_entry = (chunks + att::kGapChunks) * n_groups;
    // rows of one head and prefixes of chunks are counted in 32 bits
    if (rows >= (int64_t(1) << 31) || entries >= (int64_t(1) << 31) ||
        per_entry >= (int64_t(1) << 30) ||
        cache->num_slots * n_kv_heads >= (int64_t(1) << 32))
        return ATTN_ERR_SHAPE;
    plan->row_blocks = (int)row_blocks;
    plan->entries = (int)entries;
    plan->per_launch = (int)std::max<int64_t>(
        1, std::min<int64_t>(std::min<int64_t>(entries, parts ? att::kPartEntries : att::kMaxEntries),
                             (int64_t(1) << 30) / per_entry));
    const int per_sm = cache->dtype != ATTN_KV_BF16 ? 3 : head_dim == 64 ? 3 : 2;
    const int64_t needed = ((int64_t)plan->per_launch * (usual + att::kGapChunks) * n_groups +
                            att::kMinChunks - 1) / att::kMinChunks;
    plan->grid = (int)std::max<int64_t>(
        1, std::min<int64_t>(needed, (int64_t)per_sm * device_sm_count()));
    // Shares taken by whoever is free, two a CTA: CTAs of a grid whose SMs are partly taken by the
    // launch beside it start late, and one share each left the last with a whole one (64 requests of
    // 64 to 1,024 own keys 59.5 us, so 47.8; 256 of 32 to 256 172 and 155; 16 of up to 2,000 30.9
    // and 32.2)
    plan->pieces = parts ? 2 * plan->grid : plan->grid;
    const size_t units = (size_t)plan->per_launch * n_groups,
                 slots = (units + plan->pieces) * plan->heads;
    // How many CTAs a unit spans when all are as long as they can be: past
    // kKernelParts the merge kernel adds the parts up (else the kernel keeps to them)
    const int64_t share = std::max<int64_t>(
        att::kMinChunks, (int64_t)units * (usual + att::kGapChunks) / plan->grid);
    plan->merge = parts || usual / share + 1 > att::kKernelParts;
    // the counters are attn_decode's (zero between calls: one workspace serves both),
    // the rest lies behind them
    DecodePlan dp;
    plan_decode(cache, batch, q_rows, n_q_heads, n_kv_heads, head_dim, max_seq_len, window, &dp);
    plan->count_offset = dp.counter_offset;
    plan->parts_offset = (dp.counter_bytes + 255) & ~size_t(255);
    plan->lse_offset = (plan->parts_offset + units * sizeof(int2) + 255) & ~size_t(255);
    plan->o_offset = (plan->lse_offset + slots * rb * sizeof(float) + 255) & ~size_t(255);
    plan->workspace = plan->o_offset + slots * rb * (size_t)head_dim * sizeof(float);
    plan->launches = (plan->entries + plan->per_launch - 1) / plan->per_launch * (plan->merge ? 2 : 1);
    return ATTN_OK;
}

namespace att {

// The kernels' parameters but for the launch's entries.
Params params_of(const AttendPlan &plan, const void *q, const attn_kv_cache *cache,
                 const int32_t *seq_lens, const int32_t *positions, int q_rows, int max_seq_len,
                 int window, int sinks, int n_q_heads, int n_kv_heads, float scale, void *out,
                 void *workspace, int32_t *err) {
    Params p = {};
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
    if (cache->kind == ATTN_CACHE_PAGED && cache->block_size % att::kChunk == 0) {
        // n / d as n m / 2^(28 + s), m = floor(2^(28 + s) / d) + 1, 2^s >= d: m is at most 1
        // too large, so the quotient at most n / 2^(28 + s) < 1 / d, and its floor is exact
        const uint32_t d = (uint32_t)(cache->block_size / att::kChunk);
        while ((1u << p.page_shift) < d) ++p.page_shift;
        p.page_mul = (uint32_t)((uint64_t(1) << (28 + p.page_shift)) / d + 1);
        p.page_chunks = (int)d;
    }
    p.head_major = cache->layout == ATTN_LAYOUT_BHSD;
    p.block_table = cache->kind == ATTN_CACHE_PAGED ? cache->block_table : nullptr;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.q_rows = q_rows;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = n_kv_heads;
    p.n_groups = n_kv_heads / plan.heads;
    p.group = n_q_heads / n_kv_heads;
    p.rows = q_rows * p.group;
    p.row_blocks = plan.row_blocks;
    p.window = window;
    p.sinks = window > 0 ? sinks : 0;  // without a window every key is visible
    p.max_seq_len = max_seq_len;
    p.grid = p.pieces = plan.grid;
    p.scale_log2 = scale * 1.4426950408889634f;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.ws_parts = reinterpret_cast<int2 *>(ws + plan.parts_offset);
    p.ws_count = plan.merge ? nullptr : reinterpret_cast<int32_t *>(ws + plan.count_offset);
    p.ws_lse = reinterpret_cast<float *>(ws + plan.lse_offset);
    p.ws_o = reinterpret_cast<float *>(ws + plan.o_offset);
    p.err = err;
    return p;
}

// One of the kernels for a cache's format, the plan's rows and its heads
template <typename F>
int by_format(const attn_kv_cache *cache, F go) {
    if (cache->dtype == ATTN_KV_BF16) return go(std::integral_constant<int, kBF16>{});
    if (cache->dtype == ATTN_KV_INT8_SCALED) return go(std::integral_constant<int, kINT8>{});
    return go(std::integral_constant<int, kE4M3>{});
}

// The launch of p.n_entries entries from p.e0 on, and of the merge kernel.
int run(const Params &p, const AttendPlan &plan, const attn_kv_cache *cache, int head_dim,
        cudaStream_t stream) {
    return by_format(cache, [&](auto fmt_c) -> int {
        constexpr int F = decltype(fmt_c)::value;
        if (head_dim == 128)
            return plan.mt == 0 ? launch<F, 128, 0, 1>(p, plan.merge, stream)
                                : launch<F, 128, 1, 1>(p, plan.merge, stream);
        if (plan.mt == 0)
            return plan.heads == 1 ? launch<F, 64, 0, 1>(p, plan.merge, stream)
                                   : launch<F, 64, 0, 2>(p, plan.merge, stream);
        if (plan.heads == 1) return launch<F, 64, 1, 1>(p, plan.merge, stream);
        if constexpr (F != kBF16) return launch<F, 64, 1, 2>(p, plan.merge, stream);
        return ATTN_ERR_UNSUPPORTED;
    });
}

// ... of launch_attend_parts
template <int FMT, int HD, int MT>
int run_parts(const Params &p, int heads, cudaStream_t stream) {
    if constexpr ((FMT == kBF16 || HD == 64) && MT == 0)
        if (heads == 4) return launch<FMT, HD, MT, 4, kPartEntries>(p, false, stream);
    return heads == 2 ? launch<FMT, HD, MT, 2, kPartEntries>(p, false, stream)
                      : launch<FMT, HD, MT, 1, kPartEntries>(p, false, stream);
}

}  // namespace att

int launch_attend(const AttendPlan &plan, const void *q, const attn_kv_cache *cache,
                  const int32_t *seq_lens, const int32_t *positions, int q_rows, int max_seq_len,
                  int window, int sinks, int n_q_heads, int n_kv_heads, int head_dim, float scale,
                  void *out, void *workspace, int32_t *err, cudaStream_t stream) {
    att::Params p = att::params_of(plan, q, cache, seq_lens, positions, q_rows, max_seq_len, window,
                                   sinks, n_q_heads, n_kv_heads, scale, out, workspace, err);
    for (p.e0 = 0; p.e0 < plan.entries; p.e0 += plan.per_launch) {
        p.n_entries = std::min(plan.per_launch, plan.entries - p.e0);
        if (int rc = att::run(p, plan, cache, head_dim, stream); rc != ATTN_OK) return rc;
    }
    return ATTN_OK;
}

int launch_attend_parts(const AttendPlan &plan, int e0, const int32_t *from, int from_cap,
                        const void *q, const attn_kv_cache *cache, const int32_t *seq_lens,
                        const int32_t *positions, int q_rows, int max_seq_len, int window,
                        int n_q_heads, int n_kv_heads, int head_dim, float scale, void *out,
                        void *workspace, int32_t *err, cudaStream_t stream, bool late_wait,
                        AttendParts *parts) {
    att::Params p = att::params_of(plan, q, cache, seq_lens, positions, q_rows, max_seq_len, window,
                                   0, n_q_heads, n_kv_heads, scale, out, workspace, err);
    p.from = from;
    p.from_cap = from_cap;
    p.late_wait = late_wait;
    p.next = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + plan.count_offset);
    p.pieces = plan.pieces;
    p.e0 = e0;
    p.n_entries = std::min(plan.per_launch, plan.entries - e0);
    parts->o = p.ws_o;
    parts->lse = p.ws_lse;
    parts->parts = p.ws_parts;
    parts->next = p.next;
    parts->rb = plan.mt == 0 ? 8 : 16;
    parts->heads = plan.heads;
    parts->row_blocks = plan.row_blocks;
    parts->e0 = e0;
    parts->n_entries = p.n_entries;
    parts->held = cache->dtype == ATTN_KV_BF16 ? 0.f : att::kWeightLog2;
    return att::by_format(cache, [&](auto fmt_c) -> int {
        constexpr int F = decltype(fmt_c)::value;
        if (head_dim == 128)
            return plan.mt == 0 ? att::run_parts<F, 128, 0>(p, plan.heads, stream)
                                : att::run_parts<F, 128, 1>(p, plan.heads, stream);
        return plan.mt == 0 ? att::run_parts<F, 64, 0>(p, plan.heads, stream)
                            : att::run_parts<F, 64, 1>(p, plan.heads, stream);
    });
}

}  // namespace gqa
